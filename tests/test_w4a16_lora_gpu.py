"""gptq_w4a16_lora against its definition in float64: exact where every value
is representable, within the fp32 sums' bound elsewhere."""
import numpy as np
import pytest
import torch

from post_weight_quantization_11_b200 import gptq as G
from tests import decode_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _t(a):
    if a is None:
        return None
    a = np.ascontiguousarray(a)
    return torch.from_numpy(a.view(np.int32) if a.dtype == np.uint32 else a).to(DEV)


def _case(seed, T, m, d, g, r, n, act, exact=False, ids=None):
    rng = np.random.default_rng(seed)
    lay = R.packed_layer(rng, m, d, g, act, exact)
    if exact:
        x = rng.integers(-3, 4, (T, d)).astype(np.float16)
        a = rng.integers(-1, 2, (n, r, d)).astype(np.float16)
        b = rng.integers(-2, 3, (n, m, r)).astype(np.float16)
        sc = (2.0 ** -rng.integers(0, 3, n)).astype(np.float32)
    else:
        x = rng.standard_normal((T, d)).astype(np.float32)
        x[:, rng.permutation(d)[: max(1, d // 100)]] *= 40.0
        x = x.astype(np.float16)
        a = (rng.standard_normal((n, r, d)) * 0.05).astype(np.float16)
        b = (rng.standard_normal((n, m, r)) * 0.05).astype(np.float16)
        sc = rng.uniform(-2, 2, n).astype(np.float32)
    if ids is None:
        ids = rng.integers(-1, n, T)
    return x, lay, a, b, sc, np.asarray(ids, np.int32)


def _run(x, lay, a, b, sc, ids, **kw):
    return G.gptq_w4a16_lora(_t(x), _t(lay["qw"]), _t(lay["sc"]), _t(lay["qz"]), _t(a), _t(b),
                             _t(ids), _t(sc), lay["g"], _t(lay["perm"]), **kw)


SHAPES = [(1, 64, 128, 32, 8, 1, False), (1, 301, 256, 128, 16, 3, True),
          (2, 77, 1152, 64, 24, 5, False), (3, 16, 384, 96, 8, 2, True),
          (5, 130, 4096, -1, 64, 4, False), (7, 33, 2304, 256, 16, 9, True),
          (8, 129, 14336, 128, 16, 8, True), (9, 50, 640, 32, 40, 3, False),
          (17, 260, 1024, 64, 8, 4, True), (33, 64, 4224, 128, 128, 3, False),
          (64, 100, 512, 512, 256, 2, False), (93, 143, 768, 128, 16, 30, True),
          (200, 257, 896, 64, 16, 7, False), (300, 40, 256, 32, 8, 2, True),
          (16, 200, 5632, 64, 16, 5, True), (12, 65, 32768, 128, 8, 2, False),
          (40, 63, 960 * 2, 96, 24, 4, True), (20, 4100, 256, 64, 48, 3, True)]


@pytest.mark.parametrize("T,m,d,g,r,n,act", SHAPES)
def test_exact_on_representable_values(T, m, d, g, r, n, act):
    """Integers and powers of two: every sum is exact in fp32, so y is equal bit
    for bit (a wrong code, row, rank, adapter or permutation entry shows)."""
    c = _case(100 + T + d, T, m, d, g, r, n, act, exact=True)
    y = _run(*c).cpu().numpy()
    ref, _ = R.lora(*c)
    assert np.array_equal(y.astype(np.float64), ref)


@pytest.mark.parametrize("T,m,d,g,r,n,act", SHAPES)
def test_general_within_the_sums_bound(T, m, d, g, r, n, act):
    c = _case(200 + T + d, T, m, d, g, r, n, act)
    y = _run(*c).cpu().numpy()
    ref, bound = R.lora(*c)
    assert (np.abs(y - ref) <= bound).all()


def test_adapter_ids():
    """No adapter anywhere; one adapter for all; alternating; the last one."""
    for ids in ([-1] * 6, [2] * 6, [0, 1, 0, 1, -1, 1], [2, -1, 2, 0, 0, 2]):
        c = _case(7, 6, 90, 512, 128, 16, 3, False, exact=True, ids=ids)
        assert np.array_equal(_run(*c).cpu().numpy().astype(np.float64), R.lora(*c)[0])


def test_without_adapters_equals_the_packed_product():
    x, lay, a, b, sc, ids = _case(8, 5, 200, 1024, 128, 16, 2, True, exact=True, ids=[-1] * 5)
    y = _run(x, lay, a[:0], b[:0], sc[:0], ids)
    y0 = G.gptq_w4a16_matmul(_t(x), _t(lay["qw"]), _t(lay["sc"]), _t(lay["qz"]), 128,
                             _t(lay["perm"]))
    assert torch.equal(y, y0)


def test_bad_indices_are_recorded():
    c = list(_case(9, 4, 64, 256, 64, 8, 2, True, exact=True, ids=[0, 2, -2, 1]))
    G.gptq_device_status()
    y = _run(*c)
    torch.cuda.synchronize()
    assert G.gptq_device_status() == 0x201
    assert np.array_equal(y.cpu().numpy().astype(np.float64), R.lora(*c)[0])   # handled as -1
    c[1]["perm"][3] = 256
    _run(*c)
    torch.cuda.synchronize()
    assert G.gptq_device_status() == 0x201
    assert G.gptq_device_status() == 0


def test_runs_are_equal_bit_for_bit():
    c = _case(10, 40, 1000, 2048, 128, 16, 5, False)
    assert torch.equal(_run(*c), _run(*c))


def test_infinite_activations_stay_in_their_row():
    c = list(_case(11, 4, 64, 512, 128, 8, 2, False, exact=True))
    c[0][1, 5] = np.inf
    y = _run(*c).cpu().numpy()
    assert not np.isfinite(y[1]).all()
    keep = [0, 2, 3]
    ref, _ = R.lora(c[0][keep], c[1], c[2], c[3], c[4], c[5][keep])
    assert np.array_equal(y[keep].astype(np.float64), ref)


def test_graph_replay_other_stream_and_given_buffers():
    c = _case(12, 3, 500, 1024, 64, 16, 4, True)
    x = _t(c[0])
    lay = {k: _t(c[1][k]) for k in ("qw", "sc", "qz", "perm")}
    a, b, sc, ids = (_t(v) for v in (c[2], c[3], c[4], c[5]))
    y = torch.full((3, 500), 7.0, device=DEV)
    ws = torch.full((G.gptq_w4a16_lora_workspace_bytes(3, 500, 1024, 64, 16),), 255, dtype=torch.uint8,
                    device=DEV)
    call = lambda: G.gptq_w4a16_lora(x, lay["qw"], lay["sc"], lay["qz"], a, b, ids, sc, 64,  # noqa
                                     lay["perm"], y, ws)
    want = call().clone()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        call()
    for k in range(2):
        ws.fill_(255 * k)
        y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    x.copy_(x.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    c2 = (c[0][::-1], *c[1:])
    ref, bound = R.lora(*c2)
    assert (np.abs(y.cpu().numpy() - ref) <= bound).all()


def test_no_rows():
    c = _case(13, 2, 64, 256, 64, 8, 2, False)
    assert _run(c[0][:0], *c[1:5], c[5][:0]).shape == (0, 64)


def test_refusals():
    x, lay, a, b, sc, ids = _case(14, 2, 64, 256, 64, 8, 2, False)
    with pytest.raises(ValueError):
        _run(x.astype(np.float32), lay, a, b, sc, ids)
    with pytest.raises(ValueError):
        _run(x, lay, a, b[:, :50], sc, ids)
    with pytest.raises(ValueError):
        _run(x, lay, a, b, sc, ids[:1])
    with pytest.raises(ValueError):
        _run(x, dict(lay, g=32), a, b, sc, ids)               # scales of other groups
    with pytest.raises(ValueError):
        G.gptq_w4a16_lora(_t(x), None, _t(lay["sc"]), _t(lay["qz"]), _t(a), _t(b), _t(ids), _t(sc), 64)
    with pytest.raises(ValueError):
        G.gptq_w4a16_lora(x, _t(lay["qw"]), _t(lay["sc"]), _t(lay["qz"]), _t(a), _t(b), _t(ids), _t(sc), 64)
    with pytest.raises(G.GptqError):
        _run(x, lay, a[:, :4], b[:, :, :4], sc, ids)          # rank 4
    with pytest.raises(G.GptqError):
        _run(x, lay, a, b, sc, ids, ws=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        _run(x, lay, a, b, sc, ids, y=torch.empty(2, 65, device=DEV))


# ---- many rows: the joining kernel on the tensor cores ---------------------

@pytest.mark.parametrize("d,g,r,m", [(128, 64, 8, 1), (128, -1, 40, 129), (384, 128, 256, 300),
                                     (640, 64, 72, 31)])
@pytest.mark.parametrize("ids", ["none", "one", "alternating", "runs", "all different"])
def test_adapter_ids_of_many_rows(d, g, r, m, ids):
    T, n = 37, 40
    ids = {"none": [-1] * T, "one": [39] * T, "alternating": [3, -1, 3, 0] * 9 + [1],
           "runs": [5] * 11 + [-1] * 2 + [6] * 13 + [5] * 11, "all different": list(range(T))}[ids]
    c = _case(20 + d + r, T, m, d, g, r, n, d == 384, exact=True, ids=ids)
    assert np.array_equal(_run(*c).cpu().numpy().astype(np.float64), R.lora(*c)[0])


def test_scalings_far_apart_in_many_rows():
    """The parts of t are taken after a power of two of each row: scalings far outside
    fp16's range lose nothing."""
    c = list(_case(21, 30, 90, 512, 64, 16, 6, False, ids=list(range(6)) * 5))
    c[4] = np.array([1e30, -3e-30, 7e4, 1e-9, 1.0, 0.0], np.float32)
    y = _run(*c).cpu().numpy()
    ref, bound = R.lora(*c)
    assert (np.abs(y - ref) <= bound).all()


def test_infinities_stay_in_their_rows_of_many():
    """An infinite activation, and infinite elements of one adapter's A and B: the rows
    that have nothing to do with them are as without."""
    ids = [0, 1, 2, -1] * 6
    c = list(_case(22, 24, 64, 512, 128, 8, 3, False, exact=True, ids=ids))
    clean = [v.copy() if isinstance(v, np.ndarray) else v for v in c]
    c[0][4, 5] = np.inf                                    # a row of adapter 0
    c[2][1, 3, 7] = np.inf
    c[3][2, 9, 2] = np.inf
    y = _run(*c).cpu().numpy()
    assert not np.isfinite(y[4]).all() and not np.isfinite(y[1]).any() and not np.isfinite(y[2, 9])
    keep = [t for t in range(24) if ids[t] in (0, -1) and t != 4]
    ref, _ = R.lora(*clean)
    assert np.array_equal(y[keep].astype(np.float64), ref[keep])
    two = [t for t in range(24) if ids[t] == 2]
    rows = [i for i in range(64) if i != 9]
    assert np.array_equal(y[np.ix_(two, rows)].astype(np.float64), ref[np.ix_(two, rows)])


def test_bad_indices_in_many_rows_are_recorded():
    ids = [0, 2, -2, 1] * 6
    c = list(_case(23, 24, 64, 256, 64, 8, 2, True, exact=True, ids=ids))
    G.gptq_device_status()
    y = _run(*c)
    torch.cuda.synchronize()
    assert G.gptq_device_status() == 0x201
    assert np.array_equal(y.cpu().numpy().astype(np.float64), R.lora(*c)[0])   # handled as -1


def test_graph_replay_of_many_rows_from_any_workspace():
    c = _case(24, 60, 500, 1024, 64, 24, 4, True)
    args = [_t(c[0]), _t(c[1]["qw"]), _t(c[1]["sc"]), _t(c[1]["qz"]), _t(c[2]), _t(c[3]), _t(c[5]), _t(c[4])]
    y = torch.full((60, 500), 7.0, device=DEV)
    ws = torch.full((G.gptq_w4a16_lora_workspace_bytes(60, 500, 1024, 64, 24),), 255, dtype=torch.uint8,
                    device=DEV)
    perm = _t(c[1]["perm"])
    call = lambda: G.gptq_w4a16_lora(*args, 64, perm, y, ws)                   # noqa: E731
    want = call().clone()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        call()
        call()
    for k in range(2):
        ws.fill_(255 * k)
        y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
