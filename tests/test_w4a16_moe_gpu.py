"""gptq_w4a16_moe against its definition in float64, with the bound that the
fp32 sums carry through silu and the second product."""
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


def _case(seed, T, E, k, d, f, g, act, renorm=True):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, d)).astype(np.float32)
    x[:, rng.permutation(d)[: max(1, d // 100)]] *= 20.0
    logits = (rng.standard_normal((T, E)) * 2).astype(np.float32)
    return [x.astype(np.float16), logits, k, renorm,
            R.packed_layer(rng, 2 * f, d, g, act, lead=(E,)),
            R.packed_layer(rng, d, f, g, act, lead=(E,))]


def _run(x, logits, k, renorm, a, b, **kw):
    return G.gptq_w4a16_moe(_t(x), _t(logits), _t(a["qw"]), _t(a["sc"]), _t(a["qz"]), _t(b["qw"]),
                            _t(b["sc"]), _t(b["qz"]), k, a["g"], renorm, _t(a["perm"]),
                            _t(b["perm"]), **kw)


def _check(c):
    y = _run(*c).cpu().numpy()
    ref, bound = R.moe(*c)
    assert (np.abs(y - ref) <= bound).all()
    return y


@pytest.mark.parametrize("T,E,k,d,f,g,act,renorm", [
    (1, 1, 1, 128, 128, 32, False, True), (1, 8, 2, 512, 1024, 128, False, True),
    (1, 8, 8, 256, 384, 64, True, False), (2, 4, 1, 1152, 256, 128, False, False),
    (3, 5, 3, 384, 640, -1, True, True), (7, 32, 4, 512, 1408, 64, True, False),
    (8, 3, 2, 4096, 256, 128, False, True), (9, 2, 2, 256, 4352, 32, False, True),
    (16, 6, 2, 640, 512, 128, True, True), (24, 8, 2, 512, 768, 128, False, True),
    (33, 2, 1, 256, 256, 64, False, True), (41, 64, 8, 256, 128, 32, False, True),
    (64, 4, 3, 384, 512, 128, True, False), (64, 256, 8, 128, 128, 128, False, True),
    (5, 3, 2, 640, 384, 32, True, True), (4, 2, 2, 256, 640, 64, False, False),
    (1, 2, 1, 20480, 128, 32, False, True), (8, 1, 1, 12288, 256, 128, False, True)])
def test_against_the_definition(T, E, k, d, f, g, act, renorm):
    _check(_case(300 + T + d, T, E, k, d, f, g, act, renorm))


def test_masked_logits():
    """-inf and NaN logits: never chosen; a token with too few experts uses
    those it has, a token with none gets zero; the type's lowest value is an
    ordinary logit; +inf counts as the largest finite one."""
    c = _case(1, 7, 6, 3, 256, 256, 64, False)
    lg = c[1]
    lg[0] = -np.inf
    lg[1] = [-np.inf, 1, -np.inf, -np.inf, 2, -np.inf]
    lg[2] = np.nan
    lg[3] = [np.nan, np.nan, 0.5, np.nan, -np.inf, np.nan]
    lg[4] = np.finfo(np.float32).min
    lg[5] = [0, np.inf, 3, 1, np.inf, -np.inf]
    y = _check(c)
    assert not y[0].any() and not y[2].any()
    c[3] = False
    _check(c)


def test_equal_logits_take_the_lowest_experts():
    c = _case(2, 3, 40, 4, 128, 128, 32, False)
    c[1][:] = 1.0
    c[1][1, 35] = 2.0
    c[1][2, :3] = 0.0
    _check(c)


def test_every_token_to_one_expert():
    c = _case(3, 50, 8, 1, 256, 512, 128, False)
    c[1][:, 5] = 60.0
    _check(c)


def test_large_h_keeps_its_bits():
    """h beyond fp16's range and far below it enters the second product whole."""
    c = _case(4, 4, 2, 1, 256, 384, 128, False)
    c[0][0] *= 200
    c[0][1] = (c[0][1].astype(np.float32) * 1e-3).astype(np.float16)
    _check(c)


def test_silu_of_large_negative_gates_is_zero():
    c = _case(5, 2, 2, 1, 256, 256, 128, False)
    c[0][:] = np.where(np.abs(c[0]) < 1, c[0] * 3000, c[0] * 300).astype(np.float16)
    _check(c)


def test_infinite_activations_stay_in_their_token():
    c = _case(6, 3, 3, 2, 256, 256, 64, False)
    c[0][1, 3] = np.inf
    y = _run(*c).cpu().numpy()
    ref, bound = R.moe(c[0][[0, 2]], c[1][[0, 2]], *c[2:])
    assert (np.abs(y[[0, 2]] - ref) <= bound).all()
    assert not np.isfinite(y[1]).all()


def test_runs_are_equal_bit_for_bit_and_tokens_are_independent():
    c = _case(7, 20, 6, 2, 512, 1024, 128, False)
    y = _run(*c)
    assert torch.equal(y, _run(*c))


def test_graph_replay_with_new_routes():
    """One captured call serves other routes (the routes are read on the
    device), whatever the workspace held before."""
    c = _case(8, 5, 8, 2, 256, 512, 64, True)
    a = {k: _t(c[4][k]) for k in ("qw", "sc", "qz", "perm")}
    b = {k: _t(c[5][k]) for k in ("qw", "sc", "qz", "perm")}
    x, lg = _t(c[0]), _t(c[1])
    y = torch.empty(5, 256, device=DEV)
    ws = torch.empty(G.gptq_w4a16_moe_workspace_bytes(5, 8, 2, 256, 512), dtype=torch.uint8,
                     device=DEV)
    call = lambda: G.gptq_w4a16_moe(x, lg, a["qw"], a["sc"], a["qz"], b["qw"], b["sc"],   # noqa
                                    b["qz"], 2, 64, True, a["perm"], b["perm"], y, ws)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seed in (20, 21):
        rng = np.random.default_rng(seed)
        c[1] = (rng.standard_normal((5, 8)) * 2).astype(np.float32)
        lg.copy_(torch.from_numpy(c[1]))
        ws.fill_(255)
        y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        ref, bound = R.moe(*c)
        assert (np.abs(y.cpu().numpy() - ref) <= bound).all()


def test_bad_permutation_is_recorded():
    c = _case(9, 2, 2, 1, 256, 256, 64, True)
    c[4]["perm"][:, 7] = 256
    G.gptq_device_status()
    _run(*c)
    torch.cuda.synchronize()
    assert G.gptq_device_status() == 0x201


def test_a_quantized_layer():
    """Experts that the library quantized and packed (act-order)."""
    rng = np.random.default_rng(10)
    E, d, f = 3, 256, 384
    def stack(m, n, X):
        W = torch.from_numpy((rng.standard_normal((E, m, n)) * 0.05).astype(np.float16)).to(DEV)
        routes = [torch.arange(e, X.shape[0], E, dtype=torch.int32, device=DEV) for e in range(E)]
        return G.quantize_moe_from_inputs(W, X, routes, 4, 128, act_order=True)
    X = torch.from_numpy(rng.standard_normal((900, d)).astype(np.float16)).to(DEV)
    H = torch.from_numpy(rng.standard_normal((900, f)).astype(np.float16)).to(DEV)
    lays = []
    for res in (stack(2 * f, d, X), stack(d, f, H)):
        lays.append(dict(qw=res.qweight.cpu().numpy().view(np.uint32), sc=res.scales.cpu().numpy(),
                         qz=res.qzeros.cpu().numpy(), z=res.zeros.cpu().numpy().astype(np.int64),
                         perm=res.perm.cpu().numpy(), g=128))
    x = rng.standard_normal((6, d)).astype(np.float16)
    lg = rng.standard_normal((6, E)).astype(np.float32)
    _check([x, lg, 2, True, *lays])


def test_no_tokens():
    c = _case(11, 1, 2, 1, 128, 128, 32, False)
    assert _run(c[0][:0], c[1][:0], *c[2:]).shape == (0, 128)


def test_refusals():
    c = _case(12, 2, 3, 2, 256, 128, 64, False)
    with pytest.raises(G.GptqError):
        _run(c[0], c[1], 4, *c[3:])                           # top_k > experts
    with pytest.raises(G.GptqError):
        _run(c[0], c[1], 0, *c[3:])
    with pytest.raises(ValueError):
        _run(c[0], c[1][:1], *c[2:])
    with pytest.raises(ValueError):
        _run(c[0], c[1][:, :2].copy(), *c[2:])
    with pytest.raises(ValueError):
        _run(c[0][:, :128].copy(), *c[1:])
    with pytest.raises(G.GptqError):
        _run(*c, ws=torch.empty(64, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        G.gptq_w4a16_moe(
            _t(c[0]), None, *[_t(c[i][k]) for i in (4, 5) for k in ("qw", "sc", "qz")], 2, 64)
    big = _case(13, 65, 2, 1, 128, 128, 32, False)
    with pytest.raises(G.GptqError):
        _run(*big)
