"""The variants that the norm, the MXFP4 quantizer and its mirror take for many rows, at ragged sizes, in
all types and layouts, against their 64-bit forms with the bounds of test_gpu_rmsnorm and test_gpu_mxfp4
(the quantizer and the mirror bit for bit)."""
import numpy as np
import pytest
import torch

import ops_ref as ref
import q8_block_quantized_act_gb300 as q8
from gpu_util import device_ok, ensure_built, host
from test_gpu_mxfp4 import values
from test_gpu_rmsnorm import check_blocks, make, rel_of

pytestmark = pytest.mark.gpu
ROWS = 128                       # of the 64-bit forms at a time


@pytest.mark.parametrize("m,k,kind", [(1301, 4096, "f16"), (1301, 4096, "bf16"), (2501, 4096, "f32"), (2494, 4096, "f32"),
                                      (5003, 1280, "bf16")])
def test_quantizer_of_many_rows(m, k, kind):
    """Four rows a thread; rows beyond m in the last scale tile."""
    ensure_built()
    x = values(m, k, 3, kind)
    x[m - 1, 5] = float("inf")
    parts = [ref.mxfp4_quantize(ref.f64(p)) for p in x.split(ROWS)]
    byte, code = (np.concatenate(p) for p in zip(*parts))
    wide = torch.full((m, k + 16), float("nan"), dtype=x.dtype, device="cuda")
    wide[:, 8:8 + k] = x.cuda()
    codes = torch.full((m + 1, k // 2), 9, dtype=torch.uint8, device="cuda")
    scales = torch.full((len(ref.tile_scales(byte)),), 9, dtype=torch.uint8, device="cuda")
    q8.quantize_mxfp4(wide[:, 8:8 + k], out=(codes[:m], scales))
    device_ok()
    assert np.array_equal(host(codes[:m]), ref.pack_codes(code)) and bool((codes[m] == 9).all())
    assert np.array_equal(host(scales), ref.tile_scales(byte))


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,k", [(1301, 4096), (611, 2304), (4098, 1280)])
def test_mirror_of_many_rows(m, k, kind):
    """Four rows a thread, the last ones fewer."""
    ensure_built()
    rng = np.random.Generator(np.random.PCG64(m))
    code = rng.integers(0, 16, (m, k), dtype=np.uint8)
    byte = rng.integers(0, 255, (m, k // 32), dtype=np.uint8)
    out = torch.full((m + 1, k), 7.0, dtype=ref.TYPES[kind], device="cuda")
    q8.dequant_mxfp4(torch.from_numpy(ref.pack_codes(code)).cuda(), torch.from_numpy(ref.tile_scales(byte)).cuda(), out=out[:m])
    device_ok()
    with np.errstate(over="ignore"):
        want = torch.from_numpy(ref.mxfp4_values(byte, code).astype(np.float32)).to(ref.TYPES[kind])
    assert torch.equal(out[:m].cpu(), want) and bool((out[m] == 7.0).all())


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,k", [(3101, 8192), (3101, 4096), (1500, 8192)])
def test_norm_of_many_rows(m, k, kind):
    ensure_built()
    x, r, w = make(m, k, kind, seed=m)
    xc, rc, wc = x.cuda(), r.cuda(), w.cuda()
    s, y = torch.empty_like(xc), torch.empty_like(xc)
    q, d = q8.rmsnorm_q8_1(xc, wc, 1e-5, residual=rc, residual_out=s, y=y)
    s2, y2 = torch.empty_like(xc), torch.empty_like(xc)
    qh, dt = q8.rmsnorm_q8_1_mmq(xc, wc, 1e-5, residual=rc, residual_out=s2, y=y2)
    alone = q8.rmsnorm(xc, wc, 1e-5, residual=rc)
    bare, bare_d = q8.rmsnorm_q8_1_mmq(xc)                       # neither weight nor residual
    device_ok()
    assert torch.equal(s2, s) and torch.equal(y2, y) and torch.equal(alone, y)
    assert torch.equal(qh.view(torch.float16).float(), q.float())
    assert torch.equal(dt[:, :m].t().contiguous().view(torch.int32), d.view(torch.int32))
    for a in range(0, m, ROWS):
        b = slice(a, min(a + ROWS, m))
        s_ref, y64 = ref.rmsnorm(x[b], r[b], w, 1e-5)
        assert torch.equal(s[b].cpu(), s_ref)
        tol = (rel_of(k) + ref.HALF_ULP[kind] * 1.001) * np.abs(y64) + 2.0 ** -25 * (kind == "f16")
        assert np.all(np.abs(ref.f64(y[b]) - y64) <= tol)
        check_blocks(host(q[b]).astype(np.float64), host(d[b]).astype(np.float64), y64, k)
        _, y64 = ref.rmsnorm(x[b], None, None, 1e-6)
        check_blocks(ref.f64(bare[b].view(torch.float16)), host(bare_d[:, b]).T.astype(np.float64), y64, k)
