"""MXFP4 quantization, mirror, scale tiling and product vs their 64-bit forms.

The quantizer and the mirror are exact rules: bit for bit.  The product: |y - y64| <= 1e-5 * S,
S = sum |w x| (f32 accumulation in any order, the bound that the Q8_0 products are held to), plus
the output type's rounding (relative, and 2^-25 absolute where binary16 is subnormal)."""
import numpy as np
import pytest
import torch

import ops_ref as ref
import q8_block_quantized_act_gb300 as q8
from gpu_util import cuda, device_ok, ensure_built, host

pytestmark = pytest.mark.gpu
RTOL = 1e-5


def values(m, k, seed, kind="f32", spread=4.0):
    rng = np.random.Generator(np.random.PCG64(seed))
    x = rng.standard_normal((m, k)) * np.exp(rng.uniform(-spread, spread, (m, k // 32))).repeat(32, 1)
    return torch.from_numpy(x).to(ref.TYPES[kind])


def matrix(n, k, seed, lo=100, hi=140):
    """Every code, random scale bytes: (codes [n][k], bytes [n][k/32], packed, tiled) on the host."""
    rng = np.random.Generator(np.random.PCG64(seed))
    code = rng.integers(0, 16, (n, k), dtype=np.uint8)
    byte = rng.integers(lo, hi, (n, k // 32), dtype=np.uint8)
    return code, byte, ref.pack_codes(code), ref.tile_scales(byte)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,k", [(1, 256), (3, 4096), (128, 512), (129, 1280), (700, 768), (2, 65536)])
def test_quantize_bit_exact(m, k, kind):
    ensure_built()
    x = values(m, k, 1, kind)
    byte, code = ref.mxfp4_quantize(ref.f64(x))
    codes, scales = q8.quantize_mxfp4(x.cuda())
    device_ok()
    assert np.array_equal(host(codes), ref.pack_codes(code))
    assert np.array_equal(host(scales), ref.tile_scales(byte))      # the padding's bytes are 0


def edge_blocks():
    g = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]                      # every tie
    rows = []
    for scale in (1.0, 2.0 ** -20, 2.0 ** 100, 2.0 ** -126, 2.0 ** -140, 2.0 ** 125):
        r = np.zeros(256)
        r[:14] = [v * s for v in g for s in (1, -1)]
        r[14] = 4.0                                                  # E = 0 for this block
        r[32:64] = 7.99                                              # saturates at 6
        r[64] = -0.0
        r[96] = 1.9999999                                            # E of the next lower power
        r[128] = -2.0
        r[160:168] = np.nextafter(np.float32(5.0), np.float32(6.0))  # just above a tie
        r[160 + 8] = 4.0
        r[192:200] = np.nextafter(np.float32(0.25), np.float32(0.0))
        r[200] = 4.0
        rows.append(r * scale)
    with np.errstate(over="ignore"):
        x = np.array(rows).astype(np.float32)
    x[5, :14] = 0                                                    # keep finite what must be
    x[~np.isfinite(x)] = np.finfo(np.float32).max
    return x


def test_quantize_edge_cases():
    ensure_built()
    x = edge_blocks()
    byte, code = ref.mxfp4_quantize(x.astype(np.float64))
    codes, scales = q8.quantize_mxfp4(cuda(x))
    device_ok()
    assert np.array_equal(host(scales), ref.tile_scales(byte))
    got = host(codes)
    got = np.stack([got & 15, got >> 4], -1).reshape(x.shape)
    assert np.array_equal(got, code)


def test_quantize_nonfinite_blocks():
    ensure_built()
    x = values(3, 512, 4).numpy().astype(np.float32)
    x[0, 40], x[1, 100], x[2, 511] = np.nan, np.inf, -np.inf
    byte, code = ref.mxfp4_quantize(x.astype(np.float64))
    assert (byte == 255).sum() == 3
    codes, scales = q8.quantize_mxfp4(cuda(x))
    y = q8.dequant_mxfp4(codes, scales, dtype=torch.float32)
    device_ok()
    assert np.array_equal(host(scales), ref.tile_scales(byte))
    want = ref.mxfp4_values(byte, code)
    assert np.array_equal(np.isnan(host(y)), np.isnan(want))
    assert np.array_equal(host(y)[~np.isnan(want)], want[~np.isnan(want)].astype(np.float32))


def test_quantize_strided_rows():
    ensure_built()
    for kind in ("f32", "f16"):
        x = values(37, 512, 6, kind)
        wide = torch.zeros((37, 512 + 16), dtype=x.dtype, device="cuda")
        wide[:, 8:520] = x.cuda()
        a, b = q8.quantize_mxfp4(x.cuda()), q8.quantize_mxfp4(wide[:, 8:520])
        device_ok()
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
def test_dequant_every_code_and_scale(kind):
    """All 16 codes under every scale byte, each value rounded once to the type."""
    ensure_built()
    byte = np.arange(256, dtype=np.uint8).reshape(32, 8)
    code = np.tile(np.arange(16, dtype=np.uint8), (32, 16))
    y = q8.dequant_mxfp4(cuda(ref.pack_codes(code)), cuda(ref.tile_scales(byte)), dtype=ref.TYPES[kind])
    device_ok()
    # exact in f64; f32 holds every one but 2^128 and above; then one rounding
    with np.errstate(over="ignore"):
        want = torch.from_numpy(ref.mxfp4_values(byte, code).astype(np.float32)).to(ref.TYPES[kind])
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(y.cpu()), nan)
    assert torch.equal(y.cpu()[~nan], want[~nan])


@pytest.mark.parametrize("m,k", [(1, 256), (130, 1280), (384, 512)])
def test_tile_scales(m, k):
    ensure_built()
    byte = np.random.Generator(np.random.PCG64(3)).integers(0, 256, (m, k // 32), dtype=np.uint8)
    got = q8.tile_mxfp4_scales(cuda(byte))
    device_ok()
    assert np.array_equal(host(got), ref.tile_scales(byte))


def check_product(y, wv, xv, kind):
    y64 = xv @ wv.T
    S = np.abs(xv) @ np.abs(wv).T
    err = np.abs(ref.f64(y) - y64)
    tol = RTOL * S + ref.HALF_ULP[kind] * (np.abs(y64) + RTOL * S) * (kind != "f32") + 2.0 ** -25 * (kind == "f16")
    assert np.all(err <= tol), float((err / np.where(tol > 0, tol, 1)).max())


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,n,k", [(1, 1, 256), (1, 4096, 4096), (2, 77, 512), (8, 5152, 1280), (15, 129, 256),
                                   (16, 128, 4096), (17, 300, 2304), (33, 1000, 512), (64, 257, 1024),
                                   (65, 640, 8192), (128, 384, 256), (129, 130, 768), (191, 500, 512),
                                   (193, 1025, 1280), (300, 5152, 512), (700, 900, 1024), (1, 20493, 256),
                                   (1024, 2500, 768), (1, 33, 65536),
                                   (131, 4096, 1280), (300, 1000, 8192), (60, 1432, 2560), (100, 300, 4096),
                                   (16, 20480, 512), (193, 300, 2048), (130, 20480, 256), (12, 200, 20480)])
def test_product_matches_64_bits(m, n, k, kind):
    """Every code and spread-out scales in both operands, straight from their packed form."""
    ensure_built()
    wc, wb, wp, wt = matrix(n, k, 10 + n, 100, 124)
    xc, xb, xp, xt = matrix(m, k, 20 + m, 124, 130)
    y = q8.gemm_mxfp4_preq(cuda(wp), cuda(wt), cuda(xp), cuda(xt), dtype=ref.TYPES[kind])
    device_ok()
    assert y.shape == (m, n) and y.dtype == ref.TYPES[kind]
    check_product(y, ref.mxfp4_values(wb, wc), ref.mxfp4_values(xb, xc), kind)


@pytest.mark.parametrize("m,n,k", [(512, 20480, 512), (300, 20300, 256), (1100, 20480, 256), (257, 40000, 256),
                                   (200, 64448, 512), (1000, 19457, 256)])
def test_product_last_round(m, n, k):
    """Tiles that do not fill a last round of all SMs; ragged in both."""
    ensure_built()
    wc, wb, wp, wt = matrix(n, k, 30 + n, 100, 124)
    xc, xb, xp, xt = matrix(m, k, 40 + m, 124, 130)
    y = q8.gemm_mxfp4_preq(cuda(wp), cuda(wt), cuda(xp), cuda(xt), dtype=torch.bfloat16)
    device_ok()
    check_product(y, ref.mxfp4_values(wb, wc), ref.mxfp4_values(xb, xc), "bf16")


@pytest.mark.parametrize("m,n,k", [(1, 20480, 1024), (1, 20481, 4096), (7, 40000, 512), (16, 20353, 2304), (17, 20480, 768),
                                   (32, 45000, 256), (33, 20353, 1280), (64, 20480, 4096)])
def test_product_few_tokens_many_rows(m, n, k):
    """More row tiles than SMs, through both calls."""
    ensure_built()
    wc, wb, wp, wt = matrix(n, k, 70 + n, 100, 124)
    xc, xb, xp, xt = matrix(m, k, 80 + m, 124, 130)
    y = q8.gemm_mxfp4_preq(cuda(wp), cuda(wt), cuda(xp), cuda(xt), dtype=torch.float32)
    device_ok()
    check_product(y, ref.mxfp4_values(wb, wc), ref.mxfp4_values(xb, xc), "f32")
    x = values(m, k, 90 + m, "bf16").cuda()
    fused = q8.gemm_mxfp4(cuda(wp), cuda(wt), x)
    apart = q8.gemm_mxfp4_preq(cuda(wp), cuda(wt), *q8.quantize_mxfp4(x))
    device_ok()
    assert torch.equal(fused, apart)


@pytest.mark.parametrize("m,n,k", [(130, 9817, 2304), (265, 19451, 1792), (258, 20503, 1536), (70, 20355, 2816),
                                   (202, 9839, 1280), (791, 9628, 1280), (395, 13026, 2304), (193, 19483, 2304)])
def test_product_of_many_tiles(m, n, k):
    """Sizes that fill the GPU with wide tiles, k long enough for them to pay: one round and several,
    left-over tiles whole and cut, last tiles with few tokens and rows."""
    ensure_built()
    wc, wb, wp, wt = matrix(n, k, 50 + n, 100, 124)
    xc, xb, xp, xt = matrix(m, k, 60 + m, 124, 130)
    y = q8.gemm_mxfp4_preq(cuda(wp), cuda(wt), cuda(xp), cuda(xt), dtype=torch.float32)
    device_ok()
    check_product(y, ref.mxfp4_values(wb, wc), ref.mxfp4_values(xb, xc), "f32")


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,n,k", [(1, 640, 1024), (13, 333, 512), (200, 512, 768)])
def test_fused_call_is_quantize_then_product(m, n, k, kind):
    ensure_built()
    x = values(m, k, 8, kind, spread=1.0).cuda()
    _, _, wp, wt = matrix(n, k, 3)
    w, wsc = cuda(wp), cuda(wt)
    xq, xsc = q8.quantize_mxfp4(x)
    want = q8.gemm_mxfp4_preq(w, wsc, xq, xsc)
    wide = torch.zeros((m, k + 32), dtype=x.dtype, device="cuda")
    wide[:, :k] = x
    got, strided = q8.gemm_mxfp4(w, wsc, x), q8.gemm_mxfp4(w, wsc, wide[:, :k])
    device_ok()
    assert torch.equal(got.view(torch.int32), want.view(torch.int32))
    assert torch.equal(strided.view(torch.int32), want.view(torch.int32))


@pytest.mark.parametrize("m", [1, 9, 40, 150, 400])
def test_product_repeats_bit_for_bit_and_keeps_to_its_output(m):
    ensure_built()
    n, k = 391, 2048
    _, _, wp, wt = matrix(n, k, 5)
    _, _, xp, xt = matrix(m, k, 6, 120, 130)
    args = [cuda(a) for a in (wp, wt, xp, xt)]
    buf = torch.full((m + 2, n), 77.0, device="cuda")
    flat = buf.view(-1)
    lead = (n + 3) // 4 * 4                                   # a 16-byte aligned place inside
    out = flat[lead:lead + m * n].view(m, n)
    a = q8.gemm_mxfp4_preq(*args)
    for _ in range(3):
        q8.gemm_mxfp4_preq(*args, out=out)
        device_ok()
        assert torch.equal(out, a)
    assert bool((flat[:lead] == 77.0).all()) and bool((flat[lead + m * n:] == 77.0).all())


@pytest.mark.parametrize("m", [1, 40, 300])
def test_product_nan_blocks_reach_their_outputs_only(m):
    """A NaN scale makes its row's (token's) outputs NaN and no others, whatever the padding of the
    scale tiles holds."""
    ensure_built()
    n, k = 200, 512
    wc, wb, wp, _ = matrix(n, k, 5, 118, 126)
    xc, xb, xp, _ = matrix(m, k, 6, 118, 126)
    wb[7, 3] = 255
    xb[m - 1, 0] = 255
    y = q8.gemm_mxfp4_preq(cuda(wp), cuda(ref.tile_scales(wb, fill=255)), cuda(xp), cuda(ref.tile_scales(xb, fill=255)))
    device_ok()
    nan = np.isnan(host(y))
    want = np.zeros((m, n), bool)
    want[:, 7] = want[m - 1] = True
    assert np.array_equal(nan, want)
    wv, xv = ref.mxfp4_values(wb, wc), ref.mxfp4_values(xb, xc)
    keep = np.arange(n) != 7
    if m > 1:
        check_product(y[:m - 1][:, torch.from_numpy(keep).cuda()], wv[keep], xv[:m - 1], "f32")


@pytest.mark.parametrize("m,n", [(1, 200), (3, 200), (15, 20000), (200, 200)])
def test_fused_call_keeps_nonfinite_tokens_apart(m, n):
    """A NaN or an infinity in a token's activation reaches that token's outputs and no others."""
    ensure_built()
    k = 512
    _, _, wp, wt = matrix(n, k, 5)
    x = values(m, k, 9, spread=1.0)
    clean = q8.gemm_mxfp4(cuda(wp), cuda(wt), x.cuda())
    x[m - 1, 300] = float("nan") if m != 3 else float("-inf")
    y = q8.gemm_mxfp4(cuda(wp), cuda(wt), x.cuda())
    device_ok()
    assert bool(torch.isnan(y[m - 1]).all())
    assert torch.equal(y[:m - 1], clean[:m - 1])


@pytest.mark.parametrize("m", [1, 6, 200])
def test_product_of_zeros_and_of_extreme_scales(m):
    ensure_built()
    n, k = 130, 512
    wc, wb, wp, _ = matrix(n, k, 5)
    xc, xb, xp, _ = matrix(m, k, 6)
    zero = np.zeros_like(xp)
    y = q8.gemm_mxfp4_preq(cuda(wp), cuda(ref.tile_scales(wb)), cuda(zero), cuda(ref.tile_scales(xb)))
    device_ok()
    assert not host(y).any()
    wb[:], xb[:] = 20, 220                                    # 2^-107 times 2^93
    y = q8.gemm_mxfp4_preq(cuda(wp), cuda(ref.tile_scales(wb)), cuda(xp), cuda(ref.tile_scales(xb)))
    device_ok()
    check_product(y, ref.mxfp4_values(wb, wc), ref.mxfp4_values(xb, xc), "f32")


def test_product_follows_its_stream():
    """Weights rewritten and activations made on a side stream right before the calls that read them."""
    ensure_built()
    n, k = 640, 1024
    sets = [matrix(n, k, 30 + i) for i in range(3)]
    w = [(cuda(s[2]), cuda(s[3])) for s in sets]
    xs = {m: values(m, k, 40 + m, spread=1.0).cuda() for m in (1, 20, 260)}
    want = {(i, m): q8.gemm_mxfp4(*w[i], x) for i in range(3) for m, x in xs.items()}
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    cur = (torch.empty_like(w[0][0]), torch.empty_like(w[0][1]))
    got = {}
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for i in range(3):
            cur[0].copy_(w[i][0])
            cur[1].copy_(w[i][1])
            for m, x in xs.items():
                got[i, m] = q8.gemm_mxfp4(*cur, x * 1.0)
    side.synchronize()
    device_ok()
    for key in want:
        assert torch.equal(got[key], want[key]), key
