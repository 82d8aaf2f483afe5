"""The norm, MXFP4 and log-probability calls on arrays of more than 2^32 elements: the last rows
give what a call on those rows alone gives, bit for bit: these calls form a row's result from that row
alone, and the products have one step of k (no split to choose).  The norm's sum is formed in another
order for few rows, so its rows are held against the 64-bit form, with test_gpu_rmsnorm's bounds."""
import numpy as np
import pytest
import torch

import ops_ref as ref
import q8_block_quantized_act_gb300 as q8
from gpu_util import device_ok, ensure_built, host
from test_gpu_rmsnorm import check_blocks

pytestmark = pytest.mark.gpu
LAST = 384                     # rows compared: whole 128-row scale tiles


def tall(m, k, seed, dtype=torch.bfloat16):
    """Zeros with random last rows."""
    x = torch.zeros((m, k), dtype=dtype, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(seed)
    x[-LAST:] = torch.randn((LAST, k), generator=g, device="cuda").to(dtype)
    return x


def test_norm_rows_past_32_bits():
    ensure_built()
    m, k = (2 ** 32) // 4096 + LAST, 4096
    x = tall(m, k, 1)
    q, d = q8.rmsnorm_q8_1(x, residual=x)
    device_ok()
    s64 = 2 * ref.f64(x[-LAST:].cpu())
    y64 = s64 / np.sqrt((s64 ** 2).mean(-1, keepdims=True) + 1e-6)
    check_blocks(host(q[-LAST:]).astype(np.float64), host(d[-LAST:]).astype(np.float64), y64, k)
    assert not q[:LAST].any()


@pytest.mark.parametrize("stride", [1, 64])
def test_quantizer_and_mirror_past_32_bits(stride):
    """Many rows, and few rows far apart."""
    ensure_built()
    k = 4096
    m = (2 ** 32 // k if stride == 1 else 2 ** 32 // (k * stride)) // 128 * 128 + LAST
    x = tall(m, k, 2) if stride == 1 else torch.empty((m, k * stride), dtype=torch.bfloat16, device="cuda")[:, :k]
    if stride > 1:
        x.copy_(tall(m, k, 2))
    codes, scales = q8.quantize_mxfp4(x)
    y = q8.dequant_mxfp4(codes, scales, dtype=torch.bfloat16)
    cs, ss = q8.quantize_mxfp4(x[-LAST:].contiguous())
    ys = q8.dequant_mxfp4(cs, ss, dtype=torch.bfloat16)
    device_ok()
    assert torch.equal(codes[-LAST:], cs) and torch.equal(scales[-ss.numel():], ss) and torch.equal(y[-LAST:], ys)
    assert not y[:LAST].any()


@pytest.mark.parametrize("m,n", [(34048, 128896), (1, 2 ** 25 + LAST), (300, 2 ** 24 + LAST)])
def test_product_past_32_bits(m, n):
    """Outputs, weights: the last tokens' and the last weight rows' corner."""
    ensure_built()
    k = 256
    w, ws = q8.quantize_mxfp4(tall(n, k, 3))
    x = tall(max(m, LAST), k, 4)[-m:]
    y = q8.gemm_mxfp4(w, ws, x, dtype=torch.float16)
    tile = (n + 127) // 128 - (n - LAST) // 128
    first = (n - LAST) // 128 * 128                     # weights from a whole scale tile on
    t = min(m, LAST)
    part = q8.gemm_mxfp4(w[first:].clone(), ws[-tile * 1024:].clone(), x[-t:].contiguous(), dtype=torch.float16)
    device_ok()
    assert part[:, -LAST:].any() and torch.equal(y[-t:, first:], part)
    assert not y[:, :first].any()


def test_logprobs_past_32_bits():
    ensure_built()
    m, v = 2 ** 32 // 50257 + LAST, 50257
    x = tall(m, v, 5)
    tokens = torch.arange(m, dtype=torch.int32, device="cuda") % v
    got = q8.logprobs(x, tokens, top=4)
    part = q8.logprobs(x[-LAST:], tokens[-LAST:].clone(), top=4)
    device_ok()
    for a, b in zip(got, part):
        assert torch.equal(a[-LAST:], b)
    assert torch.equal(got[2][:3].cpu(), torch.arange(4, dtype=torch.int32).repeat(3, 1))
