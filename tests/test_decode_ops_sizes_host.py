"""Workspace sizes of the decode-step calls (no GPU): a buffer for the largest call of a
program serves its smaller ones."""
import pytest

from post_weight_quantization_11_b200 import build
from post_weight_quantization_11_b200 import gptq as G


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    G.load_library()


@pytest.mark.parametrize("m,d,g,r", [
    (14336, 4096, 128, 16), (4096, 4096, 128, 16), (4096, 11008, 64, 64), (4096, 14336, -1, 8), (4096, 4096, 32, 16),
    (6144, 4096, 64, 256), (1024, 8192, 128, 32), (64, 256, 128, 8), (1, 32768, 64, 8), (300, 32768, 32, 16),
    (50000, 384, 96, 8), (2560, 5120, 128, 16), (19000, 128, 64, 40)])
def test_the_adapters_workspace_grows_with_the_batch(m, d, g, r):
    last = 0
    for T in [*range(1, 700), *range(700, 6000, 97), 20000, 40000, 65535]:
        now = G.gptq_w4a16_lora_workspace_bytes(T, m, d, g, r)
        assert now >= last, (T, last, now)
        last = now


@pytest.mark.parametrize("m,d,g,r,most", [(14336, 4096, 128, 16, 4.2e6), (4096, 4096, 128, 16, 1.3e6),
                                          (4096, 11008, 64, 64, 3.5e6)])
def test_the_adapters_workspace_stays_small(m, d, g, r, most):
    """16 rows: their partial results at the slices that a plan may have, no more."""
    assert G.gptq_w4a16_lora_workspace_bytes(16, m, d, g, r) <= most


@pytest.mark.parametrize("E,k,d,f", [(8, 2, 4096, 14336), (32, 4, 2048, 1408), (64, 8, 2048, 1408), (256, 8, 7168, 2048),
                                     (1, 1, 128, 128), (4, 1, 20480, 32768), (16, 3, 5120, 8192), (2, 2, 640, 32768)])
def test_the_experts_workspace_grows_with_the_tokens(E, k, d, f):
    sizes = [G.gptq_w4a16_moe_workspace_bytes(T, E, k, d, f) for T in range(1, 65)]
    assert sizes == sorted(sizes)


@pytest.mark.parametrize("hq,hkv,D", [(32, 8, 128), (1024, 1, 64), (8, 8, 256), (21, 3, 64)])
@pytest.mark.parametrize("B", [1, 7, 8, 64, 65535])
def test_the_attentions_workspace_grows_and_stays_small(B, hq, hkv, D):
    """In queries and keys: never past the partial results of the most chunks that a
    launch is cut into (a prompt needs none of its own), 2 x 12 CTAs an SM of 148, eight
    rows each."""
    W = G.gptq_kv4_attention_workspace_bytes
    most = 2 * 12 * 148 * 8 * (D + 2) * 4 + 256
    for L in (1, 256, 257, 777, 9000, 131000, 1 << 30):
        sizes = [W(B, hq, hkv, D, n, L) for n in (1, 2, 9, 64, 1000, 8192, 100000, 1 << 24)]
        assert sizes == sorted(sizes) and sizes[-1] <= most, (L, sizes)
    for n in (1, 64, 8192, 1 << 24):
        sizes = [W(B, hq, hkv, D, n, L) for L in (1, 256, 257, 777, 9000, 131000, 1 << 30)]
        assert sizes == sorted(sizes), (n, sizes)
