"""gptq_kv4_append (codes equal to the quantizer's definition bit for bit) and
gptq_kv4_attention (against softmax attention in float64 over the held values)."""
import numpy as np
import pytest
import torch

from post_weight_quantization_11_b200 import gptq as G
from tests import decode_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _t(a):
    a = np.ascontiguousarray(a)
    return torch.from_numpy(a.view(np.int32) if a.dtype == np.uint32 else a).to(DEV)


def _table(n, rot):
    ang = np.arange(n)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def _np(c):
    return (c.k_codes.cpu().numpy().view(np.uint32), c.k_params.cpu().numpy(),
            c.v_codes.cpu().numpy().view(np.uint32), c.v_params.cpu().numpy())


# ---- append ---------------------------------------------------------------

def _rows(rng, T, heads, D, dt):
    x = rng.standard_normal((T, heads, D)) * rng.choice([0.01, 1, 30], (T, heads, 1))
    x[..., rng.permutation(D)[:2]] *= 10
    return x.astype(dt)


def _append_ref(k, v, pos, slots, table, inter, g, cache, page):
    """The cache after the call, from the definition"""
    kc, kp, vc, vp = (a.copy() for a in cache)
    D = k.shape[2]
    held = []
    for x, codes, params, place in ((R.rotate(k, pos, table, inter, np.float32), kc, kp,
                                     R.key_nibbles(D)),
                                    (v.astype(np.float32), vc, vp, R.value_nibbles(D))):
        c, s, z = R.quantize(x, g)
        val = (c.reshape(*c.shape[:-1], -1, g) - z[..., None]) * s.astype(np.float32)[..., None]
        held.append(val.reshape(c.shape).astype(np.float16))
        w = R.words(c, place)
        for t, sl in enumerate(slots):
            if sl >= 0:
                codes[sl // page, :, sl % page] = w[t]
                params[sl // page, :, sl % page, :, 0] = s[t]
                params[sl // page, :, sl % page, :, 1] = z[t]
    return (kc, kp, vc, vp), held


@pytest.mark.parametrize("dt", [np.float16, np.float32])
@pytest.mark.parametrize("T,hq,hkv,D,rot,inter,page,g", [
    (1, 4, 1, 64, 64, False, 16, 32), (5, 6, 2, 64, 32, True, 32, 64), (3, 0, 1, 128, 128, True, 16, 128),
    (37, 7, 7, 128, 64, False, 64, 32), (9, 5, 3, 128, 16, False, 16, 64), (4, 8, 2, 256, 256, False, 256, 256),
    (21, 3, 1, 256, 96, True, 16, 32), (6, 2, 2, 256, 48, False, 32, 128), (130, 4, 2, 128, 0, False, 64, 128)])
def test_append_equals_the_definition(T, hq, hkv, D, rot, inter, page, g, dt):
    rng = np.random.default_rng(T + D + rot)
    fused = _rows(rng, T, hq + 2 * hkv, D, dt)                # one projection's output
    fused[0, -1] = 0                                          # an all-zero row
    pages = T // page + 4
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    slots[T // 2] = -1 if T > 2 else slots[T // 2]
    pos = rng.integers(0, 5000, T).astype(np.int32)
    table = _table(5000, rot) if rot else None
    cache = G.KV4Cache.empty(pages, hkv, page, D, g, DEV)
    cache.k_codes.fill_(0x5a5a5a5a)
    cache.v_params.fill_(3.0)
    before = _np(cache)
    f = _t(fused.reshape(T, -1)).view(T, hq + 2 * hkv, D)
    q, k, v = f[:, :hq], f[:, hq:hq + hkv], f[:, hq + hkv:]
    qo, kv, vv = G.gptq_kv4_append(k, v, _t(pos), _t(slots), None if table is None else _t(table),
                                   cache, q=q if hq else None, interleaved=inter, values=True)
    want, held = _append_ref(fused[:, hq:hq + hkv], fused[:, hq + hkv:], pos, slots, table, inter, g,
                             before, page)
    for a, b in zip(_np(cache), want):
        assert np.array_equal(a, b)
    assert np.array_equal(kv.cpu().numpy(), held[0]) and np.array_equal(vv.cpu().numpy(), held[1])
    if hq:
        rq = R.rotate(fused[:, :hq], pos, table, inter, np.float32).astype(np.float16)
        assert np.array_equal(qo.cpu().numpy(), rq)
    # and against 64 bits: half a step of the group's scale, the fp16 rounding of the held value and
    # the fp32 roundings before it; 1.01 for the scale's own rounding (2^-11) over up to 15.5 steps
    x64 = R.rotate(fused[:, hq:hq + hkv], pos, table, inter, np.float64)
    _, s, _ = R.quantize(R.rotate(fused[:, hq:hq + hkv], pos, table, inter, np.float32), g)
    step = np.repeat(s.astype(np.float64), g, -1)
    assert (np.abs(held[0].astype(np.float64) - x64) <= 0.5 * step * 1.02 + 2.0 ** -11 * np.abs(x64)
            + 1e-6 * np.abs(x64).max(-1, keepdims=True)).all()


def test_append_equals_the_formula_in_fp32_tensors():
    """Scales, zero points and codes of 200000 groups are those that the formula in
    elementary fp32 tensor operations gives on the same GPU, to the last bit."""
    T, D, g = 12500, 128, 32
    gen = torch.Generator(device=DEV).manual_seed(31)
    x = torch.randn(T, 4, D, generator=gen, device=DEV) * 3.0
    cache = G.KV4Cache.empty(T // 16 + 1, 4, 16, D, g, DEV)
    at = torch.arange(T, device=DEV)
    G.gptq_kv4_append(x, x, None, at, None, cache)
    v = x.unflatten(-1, (D // g, g))
    lo, hi = v.amin(-1).clamp(max=0), v.amax(-1).clamp(min=0)
    s = ((hi - lo) / 15).half()
    z = torch.round(-lo / s.float()).clamp(0, 15)
    c = (torch.round(v / s.float()[..., None]) + z[..., None]).clamp(0, 15).flatten(-2)
    held = cache.v_params[at // 16, :, at % 16]
    assert torch.equal(held[..., 0], s) and torch.equal(held[..., 1].float(), z)
    place = torch.as_tensor(R.value_nibbles(D).astype(np.int64), device=DEV)
    words = cache.v_codes[at // 16, :, at % 16].long()
    got = (words[..., place // 8] >> (4 * (place % 8))) & 15
    assert torch.equal(got, c.long())


def test_append_unusual_values():
    """Infinities, NaN, rows of one sign, fp32 values beyond fp16, subnormals."""
    k = np.zeros((6, 1, 64), np.float32)
    k[0, 0, :3] = [np.inf, -1, 2]
    k[1, 0, :3] = [np.nan, 1, 2]
    k[2, 0] = np.linspace(1, 2, 64)
    k[3, 0] = -np.linspace(1, 2, 64)
    k[4, 0, :2] = [3e38, -3e38]
    k[5, 0] = np.linspace(-1e-9, 1e-9, 64)
    slots = np.arange(6, dtype=np.int64)
    cache = G.KV4Cache.empty(1, 1, 16, 64, 32, DEV)
    before = _np(cache)
    G.gptq_kv4_append(_t(k), _t(k), None, _t(slots), None, cache)
    want, _ = _append_ref(k, k, None, slots, None, False, 32, before, 16)
    for a, b in zip(_np(cache), want):
        assert np.array_equal(a, b)


def test_append_out_of_range_slots_and_positions():
    rng = np.random.default_rng(3)
    k = _rows(rng, 4, 2, 64, np.float16)
    cache = G.KV4Cache.empty(2, 2, 16, 64, 64, DEV)
    before = _np(cache)
    table = _table(10, 64)
    q_out = torch.full((4, 2, 64), 9.0, dtype=torch.float16, device=DEV)
    G.gptq_device_status()
    G.gptq_kv4_append(_t(k), _t(k), _t(np.array([0, 10, -1, 3], np.int32)),
                      _t(np.array([32, 1, 2, 3], np.int64)), _t(table), cache, q=_t(k), q_out=q_out)
    torch.cuda.synchronize()
    assert G.gptq_device_status() == 0x201
    want, _ = _append_ref(k[3:], k[3:], np.array([3]), np.array([3]), table, False, 64, before, 16)
    for a, b in zip(_np(cache), want):
        assert np.array_equal(a, b)
    assert (q_out[:3] == 9).all() and not (q_out[3] == 9).all()


def test_append_no_tokens_and_refusals():
    cache = G.KV4Cache.empty(2, 2, 16, 64, 32, DEV)
    e = torch.empty(0, 2, 64, dtype=torch.float16, device=DEV)
    z = torch.empty(0, dtype=torch.int64, device=DEV)
    G.gptq_kv4_append(e, e, None, z, None, cache)
    k = torch.zeros(2, 2, 64, dtype=torch.float16, device=DEV)
    s = torch.zeros(2, dtype=torch.int64, device=DEV)
    with pytest.raises(ValueError):
        G.gptq_kv4_append(k, k, None, s.int(), None, cache)
    with pytest.raises(ValueError):
        G.gptq_kv4_append(k, k.float(), None, s, None, cache)
    with pytest.raises(ValueError):
        G.gptq_kv4_append(k[:, :1], k[:, :1], None, s, None, cache)
    with pytest.raises(ValueError):
        G.gptq_kv4_append(k.transpose(1, 2).contiguous().transpose(1, 2), k, None, s, None, cache)
    with pytest.raises(ValueError):
        G.KV4Cache(cache.k_codes, cache.k_params, cache.v_codes, cache.v_params[:, :, :, :1])
    with pytest.raises(G.GptqError):                          # rotation of 8 elements
        G.gptq_kv4_append(k, k, s.int(), s, torch.zeros(4, 8, device=DEV), cache)
    with pytest.raises(G.GptqError):                          # head_dim 96
        G.gptq_kv4_append(torch.zeros(2, 2, 96, device=DEV), torch.zeros(2, 2, 96, device=DEV), None,
                          s, None, G.KV4Cache.empty(2, 2, 16, 96, 32, DEV))
    with pytest.raises(G.GptqError):                          # pages of 24
        G.gptq_kv4_append(k, k, None, s, None, G.KV4Cache.empty(2, 2, 24, 64, 32, DEV))


# ---- attention ------------------------------------------------------------

def _cache(rng, pages, hkv, page, D, g, spread=1.0):
    def half():
        codes = rng.integers(0, 2 ** 32, (pages, hkv, page, D // 8), dtype=np.uint32)
        s = rng.uniform(0.02, 0.3, (pages, hkv, page, D // g)) * spread
        z = rng.integers(0, 16, s.shape)
        return codes, np.stack([s, z], -1).astype(np.float16)
    kc, kp = half()
    vc, vp = half()
    return G.KV4Cache(_t(kc), _t(kp), _t(vc), _t(vp)), (kc, kp, vc, vp)


def _held(codes, params, place, table, L, page, sign):
    """values (sign -1) or magnitudes (+1) of a sequence's keys: L x hkv x D"""
    if L == 0:
        return np.zeros((0, codes.shape[1], len(place)))
    ids = table[: -(-L // page)]
    c = R.unpack(codes[ids])[..., place].transpose(0, 2, 1, 3).reshape(-1, codes.shape[1], len(place))
    p = params[ids].astype(np.float64).transpose(0, 2, 1, 3, 4)
    p = p.reshape(-1, *p.shape[2:])
    g = len(place) // p.shape[2]
    return ((c + sign * np.repeat(p[..., 1], g, -1)) * np.repeat(p[..., 0], g, -1))[:L]


def _attn_case(seed, lens, nqs, hq, hkv, D, page, g, spread=1.0, qs=1.0):
    rng = np.random.default_rng(seed)
    width = max(1, -(-max(lens + [1]) // page))
    B = len(lens)
    pages = B * width + 1
    cache, raw = _cache(rng, pages, hkv, page, D, g, spread)
    table = rng.permutation(pages)[: B * width].reshape(B, width).astype(np.int32)
    start = np.concatenate([[0], np.cumsum(nqs)]).astype(np.int32)
    q = (rng.standard_normal((start[-1], hq, D)) * qs).astype(np.float16)
    return dict(q=q, cache=cache, raw=raw, table=table, lens=np.array(lens, np.int32), start=start,
                page=page, D=D, scale=D ** -0.5)


def _attn_run(c, window=0, **kw):
    n = max(1, int(np.diff(c["start"]).max(initial=0)))
    return G.gptq_kv4_attention(_t(c["q"]), c["cache"], _t(c["table"]), _t(c["lens"]),
                                _t(c["start"]), c["scale"], window=window, max_q_len=n, **kw)


def _attn_ref(c, window=0):
    kc, kp, vc, vp = c["raw"]
    D, page = c["D"], c["page"]
    held = [[_held(codes, params, place, c["table"][b], L, page, sign)
             for b, L in enumerate(c["lens"])]
            for codes, params, place in ((kc, kp, R.key_nibbles(D)), (vc, vp, R.value_nibbles(D)))
            for sign in (-1, 1)]
    out = np.zeros(c["q"].shape)
    bound = R.attention(c["q"], held[0], held[2], held[1], held[3], c["scale"], list(c["lens"]),
                        list(c["start"]), window, out)
    return out, bound


def _attn_check(c, window=0, **kw):
    got = _attn_run(c, window, **kw).cpu().numpy().astype(np.float64)
    want, bound = _attn_ref(c, window)
    n = c["start"][-1]
    assert (np.abs(got - want)[:n] <= bound[:n]).all(), float((np.abs(got - want) / (bound + 1e-30)).max())
    return got


@pytest.mark.parametrize("lens,nqs,hq,hkv,D,page,g", [
    ([1], [1], 1, 1, 64, 16, 32), ([15], [1], 4, 1, 64, 16, 64), ([16, 17], [1, 1], 8, 2, 128, 16, 128),
    ([777], [1], 32, 8, 128, 16, 128), ([63, 64, 65, 1], [1, 1, 1, 1], 12, 3, 128, 32, 64),
    ([300, 5], [1, 1], 16, 1, 128, 64, 32), ([1000], [1], 12, 1, 256, 16, 256),
    ([130, 129], [2, 3], 14, 2, 64, 32, 32), ([40, 9, 200], [9, 9, 1], 21, 3, 64, 32, 32),
    ([257], [33], 8, 8, 128, 64, 64), ([515, 2], [4, 2], 8, 1, 256, 256, 32),
    ([5000], [1], 6, 2, 128, 16, 128), ([4096, 31], [1, 5], 40, 2, 64, 128, 64),
    ([100] * 20, [1] * 20, 4, 2, 256, 16, 64)])
@pytest.mark.parametrize("window", [0, 50])
def test_attention_against_the_definition(lens, nqs, hq, hkv, D, page, g, window):
    _attn_check(_attn_case(sum(lens) + hq, lens, nqs, hq, hkv, D, page, g), window)


def test_attention_rows_that_see_nothing():
    """A sequence of length 0, queries before the first key, no queries."""
    c = _attn_case(1, [0, 2, 40, 7], [1, 5, 0, 3], 4, 2, 64, 16, 32)
    got = _attn_check(c)
    assert not got[:4].any() and got[4:].any()
    _attn_check(c, 1)


def test_attention_of_no_keys_at_all():
    """A bound of 0 keys: the workspace and the call still agree, rows are zero."""
    c = _attn_case(14, [0, 0], [1, 1], 4, 2, 64, 16, 32)
    assert not _attn_run(c, max_seq_len=0).any()
    c["table"] = np.zeros((2, 0), np.int32)
    assert not _attn_run(c).any()


@pytest.mark.parametrize("hq,hkv", [(5, 5), (6, 2), (7, 1), (33, 3), (64, 1)])
def test_attention_head_groups(hq, hkv):
    """Groups of 1 .. 64 heads: rows that fill no tile, several tiles, many queries."""
    _attn_check(_attn_case(hq, [200, 77], [1, 13], hq, hkv, 64, 16, 64), 33)
    _attn_check(_attn_case(hq + 1, [1500], [3], hq, hkv, 128, 32, 64))


def test_attention_of_a_smaller_batch_fits_the_workspace_of_the_bounds():
    """One workspace for the bounds serves every smaller call."""
    W = G.gptq_kv4_attention_workspace_bytes
    most = W(40, 32, 8, 128, 4, 5000)
    for B in (1, 2, 7, 8, 39):
        for nq in (1, 4):
            for L in (0, 1, 255, 256, 257, 4999):
                assert W(B, 32, 8, 128, nq, L) <= most
    ws = torch.empty(most, dtype=torch.uint8, device=DEV)
    for lens in ([5000], [300, 299], [1000] * 9):
        _attn_check(_attn_case(len(lens), lens, [1] * len(lens), 32, 8, 128, 16, 128), ws=ws)


def test_attention_window_of_one_is_the_value():
    c = _attn_case(2, [70, 16], [2, 1], 8, 2, 128, 16, 64)
    got = _attn_check(c, 1)
    v = _held(c["raw"][2], c["raw"][3], R.value_nibbles(128), c["table"][1], 16, 16, -1)
    assert np.array_equal(got[2], np.repeat(v[15].astype(np.float16), 4, 0).astype(np.float64))


def test_attention_large_scores_and_small_values():
    """Scores of several hundred (one key takes all) and values near fp16's
    smallest scales keep their precision."""
    _attn_check(_attn_case(3, [333], [1], 8, 2, 128, 16, 64, qs=30.0))
    c = _attn_case(4, [900], [1], 8, 2, 128, 16, 128)
    c["raw"][3][..., 0] = (c["raw"][3][..., 0].astype(np.float64) * 10.0 ** np.random.default_rng(0).integers(
        -4, 1, c["raw"][3].shape[:-1])).astype(np.float16)
    c["cache"].v_params.copy_(_t(c["raw"][3]))
    _attn_check(c)


def test_attention_infinite_scale_outside_the_mask_is_not_read():
    """Slots behind a sequence's end and before its window may hold anything."""
    c = _attn_case(5, [20], [1], 4, 1, 64, 16, 32)
    p = c["table"][0, 1]
    c["cache"].k_params[p, :, 4:] = float("nan")
    c["cache"].v_params[p, :, 4:] = float("inf")
    c["cache"].v_params[c["table"][0, 0], :, :4] = float("nan")
    c["cache"].k_params[c["table"][0, 0], :, :4] = float("-inf")
    got = _attn_run(c, 16).cpu().numpy().astype(np.float64)
    want, bound = _attn_ref(c, 16)
    assert (np.abs(got - want) <= bound).all()


def test_attention_rows_behind_the_last_sequence_and_given_buffers():
    c = _attn_case(6, [33, 50], [1, 2], 4, 2, 64, 16, 32)
    c["q"] = np.concatenate([c["q"], c["q"][:2]])
    out = torch.full(c["q"].shape, 5.0, dtype=torch.float16, device=DEV)
    ws = torch.full((G.gptq_kv4_attention_workspace_bytes(2, 4, 2, 64, 2, 64) + 256,), 255,
                    dtype=torch.uint8, device=DEV)
    got = _attn_check(c, out=out, ws=ws)
    assert (got[3:] == 5).all()


def test_attention_bad_lengths_ranges_and_pages_are_recorded():
    c = _attn_case(7, [30, 40, 50], [1, 1, 1], 4, 2, 64, 16, 32)
    G.gptq_device_status()
    good = _attn_check(c)
    assert G.gptq_device_status() == 0
    for change in ("long", "negative", "page"):
        d = dict(c, lens=c["lens"].copy(), table=c["table"].copy())
        if change == "long":
            d["lens"][1] = 65
        elif change == "negative":
            d["lens"][1] = -1
        else:
            d["table"][1, 1] = 1 << 30
        out = torch.full(c["q"].shape, 5.0, dtype=torch.float16, device=DEV)
        got = _attn_run(d, out=out).cpu().numpy().astype(np.float64)
        assert G.gptq_device_status() == 0x201
        assert np.array_equal(got[[0, 2]], good[[0, 2]])
        if change != "page":
            assert (got[1] == 5).all()
    # a page that no key needs is not read
    d = dict(c, table=c["table"].copy())
    d["table"][0, 2:] = -5
    assert np.array_equal(_attn_check(d), good) and G.gptq_device_status() == 0


def test_attention_of_shared_pages_equals_separate_ones():
    """Two sequences with a common prefix on the same pages."""
    c = _attn_case(8, [48, 48], [1, 1], 4, 2, 64, 16, 32)
    c["table"][1] = c["table"][0]
    c["q"][1] = c["q"][0]
    got = _attn_check(c)
    assert np.array_equal(got[0], got[1])


def test_attention_runs_are_equal_and_graph_replays_new_lengths():
    c = _attn_case(9, [2000, 700, 1], [1, 1, 1], 8, 2, 128, 16, 128)
    assert torch.equal(_attn_run(c), _attn_run(c))
    q, table, lens, start = (_t(c[k]) for k in ("q", "table", "lens", "start"))
    out = torch.empty_like(q)
    ws = torch.empty(G.gptq_kv4_attention_workspace_bytes(3, 8, 2, 128, 1, 2000), dtype=torch.uint8,
                     device=DEV)
    call = lambda: G.gptq_kv4_attention(q, c["cache"], table, lens, start, c["scale"],  # noqa: E731
                                        max_seq_len=2000, out=out, ws=ws)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for new in ([1, 2000, 64], [513, 0, 1999]):
        c["lens"] = np.array(new, np.int32)
        lens.copy_(_t(c["lens"]))
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        want, bound = _attn_ref(c)
        assert (np.abs(out.cpu().numpy() - want) <= bound).all()


def test_attention_offsets_beyond_32_bits():
    """Pages whose words lie beyond 2^32 bytes and 2^31 elements of the cache."""
    pages, page, D = 70000, 256, 256                          # 2.3 GB of words a side
    cache = G.KV4Cache.empty(pages, 1, page, D, 256, DEV)
    rng = np.random.default_rng(10)
    small, raw = _cache(rng, 2, 1, page, D, 256)
    far = [pages - 1, pages - 40]
    for i, pg in enumerate(far):
        for a, b in zip((cache.k_codes, cache.k_params, cache.v_codes, cache.v_params),
                        (small.k_codes, small.k_params, small.v_codes, small.v_params)):
            a[pg].copy_(b[i])
    c = _attn_case(11, [500], [1], 4, 1, D, page, 256)
    c.update(cache=small, raw=raw, table=np.array([[0, 1]], np.int32))
    want = _attn_check(c)
    c2 = dict(c, cache=cache, table=np.array([far], np.int32))
    assert np.array_equal(_attn_run(c2).cpu().numpy().astype(np.float64), want)
    # and an append there
    k = _rows(rng, 1, 1, D, np.float16)
    G.gptq_kv4_append(_t(k), _t(k), None, _t(np.array([(pages - 1) * page + 255], np.int64)), None, cache)
    cc, s, z = R.quantize(k.astype(np.float32), 256)
    assert np.array_equal(cache.k_codes[pages - 1, :, 255].cpu().numpy().view(np.uint32),
                          R.words(cc, R.key_nibbles(D))[0])


def test_attention_refusals():
    c = _attn_case(12, [30], [1], 4, 2, 64, 16, 32)
    with pytest.raises(G.GptqError):
        _attn_run(c, max_seq_len=33)                          # beyond the table
    with pytest.raises(G.GptqError):
        _attn_run(c, -1)
    with pytest.raises(G.GptqError):
        _attn_run(dict(c, q=c["q"][:, :3]))                   # 3 heads on 2
    with pytest.raises(G.GptqError):
        _attn_run(dict(c, scale=float("nan")))
    with pytest.raises(ValueError):
        G.gptq_kv4_attention(c["q"], c["cache"], _t(c["table"]), _t(c["lens"]), _t(c["start"]), 1.0)
    with pytest.raises(ValueError):
        G.gptq_kv4_attention(_t(c["q"]), c["cache"], _t(c["table"]), c["lens"], _t(c["start"]), 1.0)
    with pytest.raises(ValueError):
        G.gptq_kv4_attention(_t(c["q"]).cpu(), c["cache"], _t(c["table"]), _t(c["lens"]),
                             _t(c["start"]), 1.0)
    with pytest.raises(ValueError):
        _attn_run(dict(c, q=c["q"].astype(np.float32)))
    with pytest.raises(ValueError):
        _attn_run(dict(c, lens=c["lens"].astype(np.int64)))
    with pytest.raises(ValueError):
        _attn_run(dict(c, table=np.zeros((2, 2), np.int32)))
    with pytest.raises(ValueError):
        _attn_run(c, out=torch.empty(1, 4, 32, dtype=torch.float16, device=DEV))


def test_append_then_attention_over_the_held_values():
    """Token by token: the attention over the cache equals attention over the
    fp16 values the append returned (themselves rounded: 2^-11 of the value)."""
    rng = np.random.default_rng(13)
    T, hq, hkv, D, page = 40, 8, 2, 128, 16
    cache = G.KV4Cache.empty(4, hkv, page, D, 64, DEV)
    order = rng.permutation(4)
    x = _rows(rng, T, hq + 2 * hkv, D, np.float32) * 0.2
    table = _t(_table(64, D))
    bt = _t(order[None].astype(np.int32))
    f = _t(x)
    for t in range(T):
        q, kv, vv = G.gptq_kv4_append(
            f[t:t + 1, hq:hq + hkv], f[t:t + 1, hq + hkv:], _t(np.array([t], np.int32)),
            _t(np.array([order[t // page] * page + t % page], np.int64)), table, cache,
            q=f[t:t + 1, :hq], values=True)
        o = G.gptq_kv4_attention(q, cache, bt, _t(np.array([t + 1], np.int32)),
                                 _t(np.array([0, 1], np.int32)), D ** -0.5)
        c = dict(q=q.cpu().numpy(), cache=cache, raw=_np(cache), table=order[None],
                 lens=[t + 1], start=[0, 1], page=page, D=D, scale=D ** -0.5)
        if t in (0, 1, 15, 16, 39):
            want, bound = _attn_ref(c)
            assert (np.abs(o.cpu().numpy() - want) <= bound).all()
            held = _held(c["raw"][0], c["raw"][1], R.key_nibbles(D), order, t + 1, page, -1)
            assert np.array_equal(held[t].astype(np.float16), kv[0].cpu().numpy())
