"""Refusals of the norm, MXFP4 and log-probability calls: by the C ABI before any CUDA call, and
by the torch helpers before they pass an address (no GPU needed, nothing is launched)."""
import pytest
import torch

import q8_block_quantized_act_gb300 as q8
from q8_block_quantized_act_gb300 import build as q8build

A = 1 << 20          # a fake, 16-byte aligned address: never dereferenced by these calls
MIS = A + 4
S0 = 0
F32, F16, BF16 = q8.Q8ACT_F32, q8.Q8ACT_F16, q8.Q8ACT_BF16


@pytest.fixture(scope="module")
def L():
    q8build.build()
    return q8.lib()


def norm(x=A, ldx=256, r=A, ldr=256, w=A, wt=F32, eps=1e-6, ro=A, ldro=256, y=A, q=A, d=A, m=2, k=256, t=F32, mmq=False):
    fn = q8.q8act_rmsnorm_q8_1_mmq if mmq else q8.q8act_rmsnorm_q8_1
    return fn(x, ldx, r, ldr, w, wt, eps, ro, ldro, y, q, d, m, k, t, S0)


def lp(x=A, ld=100, t=F32, tok=A, p=A, e=A, ids=A, tl=A, m=2, v=100, top=4):
    return q8.q8act_logprobs(x, ld, t, tok, p, e, ids, tl, m, v, top, S0)


def quant(x=A, ldx=256, t=F32, c=A, s=A, m=2, k=256):
    return q8.q8act_quantize_mxfp4(x, ldx, t, c, s, m, k, S0)


def gemm(w=A, ws=A, x=A, ldx=256, xt=F32, y=A, yt=F32, m=2, n=8, k=256, wk=A, nb=1 << 20):
    return q8.q8act_gemm_mxfp4(w, ws, x, ldx, xt, y, yt, m, n, k, wk, nb, S0)


def preq(w=A, ws=A, x=A, xs=A, y=A, yt=F32, m=2, n=8, k=256):
    return q8.q8act_gemm_mxfp4_preq(w, ws, x, xs, y, yt, m, n, k, S0)


def deq(c=A, s=A, y=A, t=F16, m=2, k=256):
    return q8.q8act_dequant_mxfp4(c, s, y, t, m, k, S0)


@pytest.mark.parametrize("call,want", [
    (lambda: norm(x=None), q8.Q8ACT_ERR_NULL),
    (lambda: norm(q=None), q8.Q8ACT_ERR_NULL),
    (lambda: norm(d=None, mmq=True), q8.Q8ACT_ERR_NULL),
    (lambda: norm(q=None, d=None, y=None), q8.Q8ACT_ERR_NULL),
    (lambda: norm(t=3), q8.Q8ACT_ERR_TYPE),
    (lambda: norm(wt=-1), q8.Q8ACT_ERR_TYPE),
    (lambda: norm(k=288, ldx=288, ldr=288, ldro=288), q8.Q8ACT_ERR_DIMS),
    (lambda: norm(m=0), q8.Q8ACT_ERR_DIMS),
    (lambda: norm(m=1 << 60), q8.Q8ACT_ERR_DIMS),
    (lambda: norm(m=1 << 23, mmq=True), q8.Q8ACT_ERR_DIMS),
    (lambda: norm(eps=-1.0), q8.Q8ACT_ERR_DIMS),
    (lambda: norm(eps=float("nan")), q8.Q8ACT_ERR_DIMS),
    (lambda: norm(ldx=255), q8.Q8ACT_ERR_DIMS),
    (lambda: norm(ldr=0), q8.Q8ACT_ERR_DIMS),
    (lambda: norm(ldro=128), q8.Q8ACT_ERR_DIMS),
    (lambda: norm(ldx=257), q8.Q8ACT_ERR_ALIGN),
    (lambda: norm(ldx=260, t=F16), q8.Q8ACT_ERR_ALIGN),
    (lambda: norm(x=MIS), q8.Q8ACT_ERR_ALIGN),
    (lambda: norm(w=MIS), q8.Q8ACT_ERR_ALIGN),
    (lambda: norm(y=MIS, mmq=True), q8.Q8ACT_ERR_ALIGN),
    (lambda: quant(x=None), q8.Q8ACT_ERR_NULL),
    (lambda: quant(s=None), q8.Q8ACT_ERR_NULL),
    (lambda: quant(t=7), q8.Q8ACT_ERR_TYPE),
    (lambda: quant(k=128, ldx=128), q8.Q8ACT_ERR_DIMS),
    (lambda: quant(m=0), q8.Q8ACT_ERR_DIMS),
    (lambda: quant(ldx=100), q8.Q8ACT_ERR_DIMS),
    (lambda: quant(ldx=258), q8.Q8ACT_ERR_ALIGN),
    (lambda: quant(c=MIS), q8.Q8ACT_ERR_ALIGN),
    (lambda: deq(y=None), q8.Q8ACT_ERR_NULL),
    (lambda: deq(t=9), q8.Q8ACT_ERR_TYPE),
    (lambda: deq(k=2 * q8.Q8ACT_MAX_K), q8.Q8ACT_ERR_DIMS),
    (lambda: deq(s=MIS), q8.Q8ACT_ERR_ALIGN),
    (lambda: q8.q8act_tile_mxfp4_scales(None, A, 2, 256, S0), q8.Q8ACT_ERR_NULL),
    (lambda: q8.q8act_tile_mxfp4_scales(A, A, 2, 300, S0), q8.Q8ACT_ERR_DIMS),
    (lambda: q8.q8act_tile_mxfp4_scales(A, MIS, 2, 256, S0), q8.Q8ACT_ERR_ALIGN),
    (lambda: gemm(w=None), q8.Q8ACT_ERR_NULL),
    (lambda: gemm(xt=5), q8.Q8ACT_ERR_TYPE),
    (lambda: gemm(yt=5), q8.Q8ACT_ERR_TYPE),
    (lambda: gemm(n=0), q8.Q8ACT_ERR_DIMS),
    (lambda: gemm(m=-1), q8.Q8ACT_ERR_DIMS),
    (lambda: gemm(k=320, ldx=320), q8.Q8ACT_ERR_DIMS),
    (lambda: gemm(wk=None), q8.Q8ACT_ERR_WORKSPACE),
    (lambda: gemm(nb=100), q8.Q8ACT_ERR_WORKSPACE),
    (lambda: gemm(ldx=255), q8.Q8ACT_ERR_DIMS),
    (lambda: gemm(x=MIS), q8.Q8ACT_ERR_ALIGN),
    (lambda: gemm(wk=MIS), q8.Q8ACT_ERR_ALIGN),
    (lambda: preq(xs=None), q8.Q8ACT_ERR_NULL),
    (lambda: preq(yt=-2), q8.Q8ACT_ERR_TYPE),
    (lambda: preq(n=1 << 40), q8.Q8ACT_ERR_DIMS),
    (lambda: preq(y=MIS), q8.Q8ACT_ERR_ALIGN),
    (lambda: lp(x=None), q8.Q8ACT_ERR_NULL),
    (lambda: lp(tok=None), q8.Q8ACT_ERR_NULL),
    (lambda: lp(p=None), q8.Q8ACT_ERR_NULL),
    (lambda: lp(ids=None), q8.Q8ACT_ERR_NULL),
    (lambda: lp(t=4), q8.Q8ACT_ERR_TYPE),
    (lambda: lp(m=0), q8.Q8ACT_ERR_DIMS),
    (lambda: lp(v=0), q8.Q8ACT_ERR_DIMS),
    (lambda: lp(v=101), q8.Q8ACT_ERR_DIMS),
    (lambda: lp(top=q8.Q8ACT_MAX_TOP + 1), q8.Q8ACT_ERR_DIMS),
    (lambda: lp(top=-1), q8.Q8ACT_ERR_DIMS),
    (lambda: lp(x=A + 2), q8.Q8ACT_ERR_ALIGN),
    (lambda: lp(e=A + 2), q8.Q8ACT_ERR_ALIGN),
])
def test_abi_refusals(L, call, want):
    assert call() == want


def test_sizes(L):
    assert q8.q8act_mxfp4_scale_bytes(1, 256) == 1024
    assert q8.q8act_mxfp4_scale_bytes(129, 4096) == 2 * 32 * 512
    assert q8.q8act_mxfp4_scale_bytes(0, 256) == 0 and q8.q8act_mxfp4_scale_bytes(4, 100) == 0
    assert q8.q8act_gemm_mxfp4_workspace_bytes(3, 256) == 512 + 1024
    assert q8.q8act_gemm_mxfp4_workspace_bytes(3, 257) == 0
    assert isinstance(q8.strerror(q8.Q8ACT_ERR_TYPE), str) and "type" in q8.strerror(q8.Q8ACT_ERR_TYPE)


def test_helpers_refuse_host_tensors(L):
    """An address of host memory never reaches a kernel."""
    x = torch.zeros((2, 256))
    u8 = torch.zeros((2, 128), dtype=torch.uint8)
    for call in (lambda: q8.rmsnorm_q8_1(x), lambda: q8.rmsnorm_q8_1_mmq(x), lambda: q8.quantize_mxfp4(x),
                 lambda: q8.dequant_mxfp4(u8, u8), lambda: q8.tile_mxfp4_scales(u8), lambda: q8.gemm_mxfp4(u8, u8, x),
                 lambda: q8.gemm_mxfp4_preq(u8, u8, u8, u8), lambda: q8.logprobs(x)):
        with pytest.raises(q8.Q8ActError) as e:
            call()
        assert e.value.rc == q8.Q8ACT_ERR_DEVICE


@pytest.mark.gpu
def test_helpers_refuse_what_the_kernels_cannot_take():
    q8build.build()
    dev = torch.device("cuda")
    x = torch.zeros((4, 512), device=dev)
    w, wsc = q8.quantize_mxfp4(x)
    i32 = torch.zeros(4, dtype=torch.int32, device=dev)
    f = torch.float16
    cases = [
        (lambda: q8.rmsnorm_q8_1(x.double()), q8.Q8ACT_ERR_TYPE),
        (lambda: q8.rmsnorm_q8_1(x.t()), q8.Q8ACT_ERR_DIMS),
        (lambda: q8.rmsnorm_q8_1(x[:, ::2]), q8.Q8ACT_ERR_DIMS),
        (lambda: q8.rmsnorm_q8_1(x[:, :511]), q8.Q8ACT_ERR_DIMS),
        (lambda: q8.rmsnorm_q8_1(x[:, 1:257]), q8.Q8ACT_ERR_ALIGN),
        (lambda: q8.rmsnorm_q8_1(x, residual=x.half()), q8.Q8ACT_ERR_TYPE),
        (lambda: q8.rmsnorm_q8_1(x, residual_out=x[:3]), q8.Q8ACT_ERR_TYPE),
        (lambda: q8.rmsnorm_q8_1(x, x[0, :256]), q8.Q8ACT_ERR_DIMS),
        (lambda: q8.rmsnorm_q8_1(x, out=(torch.empty((4, 512), dtype=torch.int8, device=dev), x)), q8.Q8ACT_ERR_DIMS),
        (lambda: q8.rmsnorm_q8_1_mmq(x, y=x.half()), q8.Q8ACT_ERR_TYPE),
        (lambda: q8.quantize_mxfp4(x.int()), q8.Q8ACT_ERR_TYPE),
        (lambda: q8.quantize_mxfp4(x, out=(w, wsc[:-1])), q8.Q8ACT_ERR_DIMS),
        (lambda: q8.dequant_mxfp4(w, wsc[:512]), q8.Q8ACT_ERR_DIMS),
        (lambda: q8.dequant_mxfp4(w, wsc, dtype=torch.int8), q8.Q8ACT_ERR_TYPE),
        (lambda: q8.gemm_mxfp4(w, wsc, x[:, :256]), q8.Q8ACT_ERR_DIMS),
        (lambda: q8.gemm_mxfp4(w, wsc, x, ws=torch.empty(16, dtype=torch.uint8, device=dev)), q8.Q8ACT_ERR_WORKSPACE),
        (lambda: q8.gemm_mxfp4(w, wsc, x, out=torch.empty((4, 5), device=dev)), q8.Q8ACT_ERR_DIMS),
        (lambda: q8.gemm_mxfp4(w, wsc, x, dtype=torch.float64), q8.Q8ACT_ERR_TYPE),
        (lambda: q8.gemm_mxfp4_preq(w, wsc, w[:, :128], wsc), q8.Q8ACT_ERR_DIMS),
        (lambda: q8.logprobs(x, i32.long()), q8.Q8ACT_ERR_TYPE),
        (lambda: q8.logprobs(x, i32[:3]), q8.Q8ACT_ERR_DIMS),
        (lambda: q8.logprobs(x, top=q8.Q8ACT_MAX_TOP + 1), q8.Q8ACT_ERR_DIMS),
        (lambda: q8.logprobs(x.to(f).t()), q8.Q8ACT_ERR_DIMS),
        (lambda: q8.logprobs(x[:0]), q8.Q8ACT_ERR_DIMS),
    ]
    for i, (call, want) in enumerate(cases):
        with pytest.raises(q8.Q8ActError) as e:
            call()
        assert e.value.rc == want, i
    torch.cuda.synchronize()
