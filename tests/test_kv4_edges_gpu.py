"""gptq_kv4_attention at the ends of its ranges: windows longer than the cache,
queries that are not finite, prompts."""
import numpy as np
import pytest
import torch

from post_weight_quantization_11_b200 import gptq as G
from tests.test_kv4_gpu import _attn_case, _attn_check, _attn_ref, _attn_run

pytestmark = pytest.mark.gpu

# (lengths, queries, q_heads, kv_heads, head_dim, page, group): in one chunk, in chunks that a
# cluster joins, in chunks that are joined through memory (few long ones, many of them)
PATHS = {"one chunk": ([200, 77], [1, 2], 8, 2, 64, 16, 32),
         "cluster": ([777], [1], 8, 2, 128, 16, 128),
         "cluster, five rows": ([1500, 600], [5, 5], 3, 3, 128, 32, 64),
         "joined": ([9000, 40], [1, 1], 4, 1, 64, 16, 64),
         "joined, five rows": ([9000], [5], 2, 2, 64, 64, 64),
         "joined, many": ([700 + 37 * i for i in range(40)], [1] * 40, 16, 8, 64, 16, 32)}


def _case(path, seed=0):
    return _attn_case(seed, *PATHS[path])


def _run(c, window=0):
    return _attn_run(c, window).cpu().numpy().astype(np.float64)


# ---- windows --------------------------------------------------------------

@pytest.mark.parametrize("window", [2 ** 63 - 1, 2 ** 62, 2 ** 31, 9000, 8999])
@pytest.mark.parametrize("path", list(PATHS))
def test_a_window_longer_than_the_sequences_is_none(path, window):
    """Whatever the caller has for 'no limit' gives what no window gives."""
    c = _case(path)
    got = _run(c, window)
    want, bound = _attn_ref(c, min(window, 1 << 30))
    assert (np.abs(got - want) <= bound).all()
    if window >= c["table"].shape[1] * c["page"]:
        assert np.array_equal(got, _run(c))


@pytest.mark.parametrize("window", [2 ** 63 - 1, 2 ** 62, 2 ** 31])
def test_a_long_window_with_more_queries_than_keys(window):
    """Rows before the first key see nothing, with any window."""
    c = _attn_case(1, [0, 2, 40, 7], [1, 5, 0, 9], 4, 2, 64, 16, 32)
    assert np.array_equal(_run(c, window), _attn_check(c))
    c = _attn_case(2, [3, 900], [9, 1], 8, 2, 128, 16, 64)
    assert np.array_equal(_run(c, window), _attn_check(c))


@pytest.mark.parametrize("page", [16, 32, 64])
@pytest.mark.parametrize("lens,nqs,window", [([100], [1], 20), ([1000, 90, 33], [1, 1, 1], 17), ([700], [5], 60),
                                             ([9000], [1], 8000)])
def test_pages_behind_the_window_are_not_read(lens, nqs, window, page):
    """Their entries may hold anything (a program that frees the pages puts -1 there), also
    where such a page ends inside the first tile of 32 keys."""
    G.gptq_device_status()
    for shift in range(0, 32, 5):
        c = _attn_case(6, [L + shift for L in lens], nqs, 4, 2, 64, page, 32)
        for b, (L, n) in enumerate(zip(c["lens"], nqs)):
            first = max(0, int(L) - n + 1 - window) // page              # of the first key that is seen
            c["table"][b, :first] = -1
        got = _run(c, window)
        assert G.gptq_device_status() == 0
        c["table"][c["table"] < 0] = 0
        want, bound = _attn_ref(c, window)
        assert (np.abs(got - want) <= bound).all()


# ---- queries that are not finite -------------------------------------------

@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("path", list(PATHS))
def test_a_query_that_is_not_finite_gives_a_row_that_is_not(path, value):
    """However the keys are split: no such row comes out as numbers, and no other row
    changes beyond its bound."""
    c = _case(path, 3)
    want, bound = _attn_ref(c)
    c["q"][0, 1, 5] = value
    got = _run(c)
    assert not np.isfinite(got[0, 1]).any()
    keep = np.ones(got.shape[:2], bool)
    keep[0, 1] = False
    assert (np.abs(got - want) <= bound)[keep].all()


def test_a_query_that_is_not_finite_and_sees_no_key_is_zero():
    c = _attn_case(4, [0, 300], [2, 1], 4, 2, 64, 16, 32)
    c["q"][:2] = np.nan
    got = _run(c)
    assert not got[:2].any() and np.isfinite(got[2]).all()


def test_an_infinite_query_whose_every_score_is_minus_infinity():
    """Rows that see one key: its score is an infinity of either sign, the row is NaN."""
    for path in PATHS:
        c = _case(path, 5)
        c["q"][0, 0, 3], c["q"][0, 1, 3] = np.inf, -np.inf
        got = _attn_run(c, 1).cpu().numpy()
        assert np.isnan(got[0, :2]).all() and np.isfinite(got[1:]).all() and np.isfinite(got[0, 2:]).all()


# ---- prompts ----------------------------------------------------------------

@pytest.mark.parametrize("window", [0, 100])
@pytest.mark.parametrize("lens,nqs,hq,hkv,D,page,g", [
    ([700, 300, 64], [500, 300, 1], 4, 2, 64, 16, 32), ([9000], [65], 4, 1, 64, 64, 64),
    ([400], [400], 3, 1, 128, 32, 128), ([260, 4000, 1], [9, 90, 1], 8, 2, 128, 16, 64), ([600], [200], 2, 2, 256, 16, 128)])
def test_prompts_in_the_workspace_asked_for(lens, nqs, hq, hkv, D, page, g, window):
    """Many row tiles a sequence, whose partial results stay inside the workspace."""
    c = _attn_case(sum(lens) + 7, lens, nqs, hq, hkv, D, page, g)
    n = G.gptq_kv4_attention_workspace_bytes(len(lens), hq, hkv, D, max(nqs), c["table"].shape[1] * page)
    space = torch.full((n + 65536,), 90, dtype=torch.uint8, device="cuda:0")
    _attn_check(c, window, ws=space[:n])
    assert (space[n:] == 90).all()
