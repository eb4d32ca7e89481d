"""KV4Cache.empty refuses groups that the cache cannot have (no GPU needed: before
anything is allocated)."""
import pytest

from post_weight_quantization_11_b200 import gptq as G


@pytest.mark.parametrize("head_dim,group_size", [(128, 48), (64, 128), (128, 0), (128, -2), (256, 96), (64, 24)])
def test_groups_that_do_not_divide_the_head_are_refused(head_dim, group_size):
    """A cache of other groups than asked for would be made (48 of 128: two of 64)."""
    with pytest.raises(ValueError, match="group_size"):
        G.KV4Cache.empty(2, 2, 16, head_dim, group_size, device="cpu")
