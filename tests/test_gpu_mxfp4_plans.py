"""Every variant of the MXFP4 product (test_mxfp4_plan.REACHED) against 64 bits, and the call that
quantizes the activation against the quantizer and the product apart, in all types and with strided rows.

|y - y64| <= 1e-5 * S, S = sum |w x|, as in test_gpu_mxfp4."""
import pytest
import torch

import ops_ref as ref
import q8_block_quantized_act_gb300 as q8
from gpu_util import device_ok, ensure_built
from test_mxfp4_plan import REACHED, SMS, plan

pytestmark = pytest.mark.gpu


def matrix(rows, k, seed, lo, hi):
    """Every code, random scale bytes: (packed codes, tiled scales, values in 64 bits)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    code = torch.randint(0, 16, (rows, k), generator=g, device="cuda", dtype=torch.uint8)
    byte = torch.randint(lo, hi, (rows, k // 32), generator=g, device="cuda", dtype=torch.uint8)
    mags = torch.tensor(ref.E2M1, device="cuda")
    v = torch.cat((mags, -mags))[code.int()] * torch.exp2(byte.double() - 127).repeat_interleave(32, 1)
    full = torch.zeros(((rows + 127) // 128 * 128, k // 32), dtype=torch.uint8, device="cuda")
    full[:rows] = byte
    tiled = full.view(-1, 4, 32, k // 128, 4).permute(0, 3, 2, 1, 4).reshape(-1)
    return code[:, 0::2] | (code[:, 1::2] << 4), tiled, v


@pytest.mark.parametrize("m,n,k", REACHED)
def test_variant(m, n, k):
    ensure_built()
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert sms != SMS or plan(m, n, k) == REACHED[m, n, k]
    w, wsc, wv = matrix(n, k, n + k, 100, 124)
    xq, xsc, xv = matrix(m, k, m + k, 124, 130)
    out = torch.full((m + 2, n + (-n % 4)), 77.0, device="cuda").view(-1)
    lead = n + (-n % 4)
    y = out[lead:lead + m * n].view(m, n)
    q8.gemm_mxfp4_preq(w, wsc, xq, xsc, out=y)
    device_ok()
    err = (y.double() - xv @ wv.T).abs()
    assert bool((err <= 1e-5 * (xv.abs() @ wv.abs().T)).all())
    assert bool((out[:lead] == 77.0).all()) and bool((out[lead + m * n:] == 77.0).all())


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,n,k", [s for s in REACHED if s[0] <= 16])
def test_quantizing_call(m, n, k, kind):
    ensure_built()
    g = torch.Generator(device="cuda").manual_seed(m * n)
    w, wsc, wv = matrix(n, k, n, 100, 124)
    x = torch.randn((m, k), generator=g, device="cuda") * torch.exp(
        2 * torch.randn((m, k // 32), generator=g, device="cuda")).repeat_interleave(32, 1)
    wide = torch.full((m, k + 72), float("nan"), dtype=ref.TYPES[kind], device="cuda")
    wide[:, 40:40 + k] = x.to(ref.TYPES[kind])
    x = wide[:, 40:40 + k]
    xq, xsc = q8.quantize_mxfp4(x)
    xv = q8.dequant_mxfp4(xq, xsc, dtype=torch.float32).double()
    apart = q8.gemm_mxfp4_preq(w, wsc, xq, xsc)
    strided, packed = q8.gemm_mxfp4(w, wsc, x), q8.gemm_mxfp4(w, wsc, x.contiguous())
    device_ok()
    assert torch.equal(strided, apart) and torch.equal(packed, apart)
    assert bool(((apart.double() - xv @ wv.T).abs() <= 1e-5 * (xv.abs() @ wv.abs().T)).all())
