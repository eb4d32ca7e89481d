"""One workspace, made for a program's largest call, behind its smaller ones."""
import numpy as np
import pytest
import torch

from post_weight_quantization_11_b200 import gptq as G
from tests import decode_ref as R
from tests import test_w4a16_moe_gpu as M
from tests.test_w4a16_lora_gpu import DEV, _case, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,d,g,r,act", [(900, 2048, 128, 16, True), (300, 1536, 32, 8, False), (64, 8192, 64, 24, False)])
def test_adapters_of_smaller_batches_in_the_largest_ones_workspace(m, d, g, r, act):
    ws = torch.empty(G.gptq_w4a16_lora_workspace_bytes(256, m, d, g, r), dtype=torch.uint8, device=DEV)
    for T in (256, 129, 128, 40, 17, 16, 9, 8, 3, 1):
        c = _case(T + d, T, m, d, g, r, 3, act, exact=True)
        ws.fill_(255)
        assert np.array_equal(_run(*c, ws=ws).cpu().numpy().astype(np.float64), R.lora(*c)[0])


def test_experts_of_fewer_tokens_in_the_largest_calls_workspace():
    E, k, d, f, g = 12, 3, 512, 1408, 64
    ws = torch.empty(G.gptq_w4a16_moe_workspace_bytes(64, E, k, d, f), dtype=torch.uint8, device=DEV)
    for T in (64, 33, 9, 7, 6, 5, 2, 1):
        c = M._case(T, T, E, k, d, f, g, T == 7)
        ws.fill_(255)
        y = M._run(*c, ws=ws).cpu().numpy()
        ref, bound = R.moe(*c)
        assert (np.abs(y - ref) <= bound).all()


def test_adapters_of_scales_beyond_32_bits():
    """A layer whose scales take more than 2^32 bytes, swept from its first row to its last
    by one CTA: every code 1, x integers, a row's scales a power of two of the row modulo 5."""
    m, d, g, T, r = 2 ** 21 + 192, 32768, 32, 113, 8
    assert G.gptq_w4a16_lora_workspace_bytes(T, m, d, g, r) < 40e9
    qw = torch.full((m, d // 8), 0x11111111, dtype=torch.int32, device=DEV)
    s = 2.0 ** -(torch.arange(m, device=DEV) % 5).float()
    sc = s.half()[:, None].expand(m, d // g).contiguous()
    qz = torch.zeros(m, d // g // 2, dtype=torch.uint8, device=DEV)
    gen = torch.Generator(device=DEV).manual_seed(5)
    x = torch.randint(-2, 3, (T, d), generator=gen, device=DEV).half()
    none = torch.full((T,), -1, dtype=torch.int32, device=DEV)
    a = torch.zeros(1, r, d, dtype=torch.float16, device=DEV)
    b = torch.zeros(1, m, r, dtype=torch.float16, device=DEV)
    y = G.gptq_w4a16_lora(x, qw, sc, qz, a, b, none, torch.ones(1, device=DEV), g)
    total = x.float().sum(1)
    wrong = sum(int((y[t] != total[t] * s).sum()) for t in range(T))
    del qw, sc, qz, b, y
    torch.cuda.empty_cache()
    assert wrong == 0
