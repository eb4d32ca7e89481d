"""gptq_w4a16_moe where an expert's tokens are staged in several chunks, and of batches
that differ in their other tokens."""
import numpy as np
import pytest

from tests import decode_ref as R
from tests.test_w4a16_moe_gpu import _case, _check, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E,k,d,f,g,act", [
    (20, 2, 1, 5120, 128, 128, False), (9, 3, 2, 8192, 256, 64, True), (17, 2, 2, 6144, 128, -1, False),
    (5, 2, 1, 16384, 128, 128, True), (13, 4, 2, 7168, 384, 32, False), (64, 2, 2, 640, 256, 128, True)])
def test_more_tokens_of_an_expert_than_are_staged_together(T, E, k, d, f, g, act):
    """Long rows of x leave room for six (d_model 5120) to one (16384) of them beside the
    ring: the expert's rows are swept once per chunk of its tokens."""
    c = _case(40 + T + d, T, E, k, d, f, g, act)
    c[1][:, 0] += 3                                           # most tokens to the first expert
    _check(c)


def test_a_tokens_result_in_any_batch():
    """A token alone, among others and among all: within its bound each time (the order of
    the sums follows the batch, so the last bits may differ)."""
    c = _case(51, 20, 6, 2, 512, 1024, 128, False)
    ref, bound = R.moe(*c)
    for pick in (*([t] for t in range(0, 20, 3)), range(5), range(3, 20), [19, 0, 7], [4] * 9, range(20)):
        pick = list(pick)
        y = _run(c[0][pick], c[1][pick], *c[2:]).cpu().numpy()
        assert (np.abs(y - ref[pick]) <= bound[pick]).all()
