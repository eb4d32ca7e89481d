"""The precision of the scores of gptq_kv4_attention: heads with outlier channels."""
import numpy as np
import pytest

from tests import decode_ref as R
from tests.test_kv4_gpu import _attn_case, _attn_run, _held, _t

pytestmark = pytest.mark.gpu


def _bound(c, want):
    """What out may be off by, from fp32 scores: every product (c - z) q is exact, the sums of
    them are chains of fewer than D / 8 + 10 fp32 additions (the matrix pipe's may be cut
    instead of rounded: two half steps each), so a score is off by

      es = scale (D / 8 + 10) 2 U sum_d |K| |q|,

    which, unlike a bound by s (c + z) |q|, does not grow with a channel in which the keys
    are small.  Then out by 2 es in every probability, 2^-20 for exp2 and the probabilities'
    two parts, the sums over the keys (L / 32 + 64 terms), and its own rounding."""
    kc, kp, vc, vp = c["raw"]
    D, page = c["D"], c["page"]
    bound = np.zeros(want.shape)
    for b, L in enumerate(c["lens"]):
        t = c["start"][b]
        V = np.abs(_held(vc, vp, R.value_nibbles(D), c["table"][b], L, page, 1))
        K = _held(kc, kp, R.key_nibbles(D), c["table"][b], L, page, -1)
        for h in range(want.shape[1]):
            hk = h // (want.shape[1] // K.shape[1])
            q = c["q"][t, h].astype(np.float64)
            es = c["scale"] * np.max(np.abs(K[:, hk]) @ np.abs(q)) * (D / 8 + 10) * 2 * R.U
            sc = c["scale"] * (K[:, hk] @ q)
            w = np.exp(sc - sc.max())
            w /= w.sum()
            rel = 2 * es + 2.0 ** -20 + (L / 32 + 64) * R.U
            bound[t, h] = 2.0 ** -11 * np.abs(want[t, h]) + 2.0 ** -25 + rel * (w @ V[:, hk]) * 1.01
    return bound


def _outliers(seed, lens, hq, hkv, D, page, g, size):
    """Keys that are 0 in two channels (code = zero point) in which the queries have
    elements of `size`"""
    c = _attn_case(seed, lens, [1] * len(lens), hq, hkv, D, page, g)
    rng = np.random.default_rng(seed + 1)
    kc, kp = c["raw"][:2]
    kp[..., 1] = rng.integers(6, 11, kp.shape[:-1])
    codes = R.unpack(kc)[..., R.key_nibbles(D)]
    far = rng.permutation(D)[:2]
    codes[..., far] = np.repeat(kp[..., 1].astype(np.float64), g, -1)[..., far]
    kc[...] = R.words(codes, R.key_nibbles(D))
    c["cache"].k_codes.copy_(_t(kc))
    c["cache"].k_params.copy_(_t(kp))
    c["q"][:, :, far] = rng.choice([-size, size], (*c["q"].shape[:2], 2))
    return c


@pytest.mark.parametrize("size", [100, 3000])
@pytest.mark.parametrize("lens,hq,hkv,D,page,g", [
    ([40], 4, 2, 64, 16, 64), ([60, 33], 5, 1, 64, 32, 32), ([50], 4, 2, 128, 16, 128),
    ([40, 64], 24, 3, 128, 16, 32), ([31], 8, 8, 256, 16, 256), ([64], 6, 1, 256, 64, 64)])
def test_scores_with_outlier_channels(lens, hq, hkv, D, page, g, size):
    c = _outliers(sum(lens) + D, lens, hq, hkv, D, page, g, size)
    got = _attn_run(c).cpu().numpy().astype(np.float64)
    want = np.zeros(got.shape)
    for b, L in enumerate(c["lens"]):
        K = _held(c["raw"][0], c["raw"][1], R.key_nibbles(D), c["table"][b], L, page, -1)
        V = _held(c["raw"][2], c["raw"][3], R.value_nibbles(D), c["table"][b], L, page, -1)
        for h in range(hq):
            sc = c["scale"] * (K[:, h // (hq // hkv)] @ c["q"][c["start"][b], h].astype(np.float64))
            w = np.exp(sc - sc.max())
            want[c["start"][b], h] = w @ V[:, h // (hq // hkv)] / w.sum()
    bound = _bound(c, want)
    assert (np.abs(got - want) <= bound).all(), float((np.abs(got - want) / bound).max())
