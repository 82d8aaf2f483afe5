"""The norm in front of a product vs its 64-bit form.

Tolerances.  The f32 sum of k squares is a sum of non-negative terms in which no term passes
through more than depth = k / 64 + 32 additions, so its relative error is below depth * 2^-24
(plus 2^-24 for each square); the square root halves it, and the division, the root, the mean and
the two products add 2^-24 each: rel = (depth / 2 + 8) * 2^-24.  A scale is then within
rel + 2^-23 of its own value, and a quant within 1/2 + 127 * 2 (rel + 2^-23) of y / d."""
import numpy as np
import pytest
import torch

import ops_ref as ref
import q8_block_quantized_act_gb300 as q8
from gpu_util import device_ok, ensure_built, host

pytestmark = pytest.mark.gpu


def rel_of(k):
    return ((k / 64 + 32) / 2 + 8) * ref.U


def make(m, k, kind, seed=0, residual=True, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((m, k), generator=g) * spread
    x[torch.rand((m, k), generator=g) < 0.01] *= 20
    r = torch.randn((m, k), generator=g) * 4 * spread if residual else None
    w = 1 + 0.1 * torch.randn(k, generator=g)
    t = ref.TYPES[kind]
    return x.to(t), None if r is None else r.to(t), w.to(t)


def check_blocks(q, d, y64, k):
    """q [m][k] integers and d [m][k/32] against the exact y."""
    rel = rel_of(k) + 2 * ref.U
    b = y64.reshape(len(y64), -1, 32)
    d64 = np.abs(b).max(-1) / 127
    assert np.all(np.abs(d - d64) <= rel * d64)
    t = np.divide(b, d64[..., None], out=np.zeros_like(b), where=d64[..., None] > 0)
    assert np.all(np.abs(q.reshape(b.shape) - t) <= 0.5 + 254 * rel)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,k,residual", [(1, 256, True), (1, 4096, True), (3, 512, False), (15, 1280, True),
                                          (133, 4096, False), (5, 65536, True), (2, 33024, False), (300, 768, True),
                                          (257, 8192, True), (1, 16640, True)])
def test_norm_matches_64_bits(m, k, kind, residual):
    ensure_built()
    x, r, w = make(m, k, kind, residual=residual)
    s_ref, y64 = ref.rmsnorm(x, r, w, 1e-5)
    xc, rc, wc = x.cuda(), None if r is None else r.cuda(), w.cuda()
    s, y = torch.empty_like(xc), torch.empty_like(xc)
    q, d = q8.rmsnorm_q8_1(xc, wc, 1e-5, residual=rc, residual_out=s, y=y)
    s2, y2 = torch.empty_like(xc), torch.empty_like(xc)
    qh, dt = q8.rmsnorm_q8_1_mmq(xc, wc, 1e-5, residual=rc, residual_out=s2, y=y2)
    device_ok()
    assert torch.equal(s.cpu(), s_ref) and torch.equal(s2, s) and torch.equal(y2, y)
    assert np.all(np.abs(ref.f64(y) - y64) <= (rel_of(k) + ref.HALF_ULP[kind] * 1.001) * np.abs(y64) + 2.0 ** -25 * (kind == "f16"))
    check_blocks(host(q).astype(np.float64), host(d).astype(np.float64), y64, k)
    # both layouts hold the same quants and scales
    assert torch.equal(qh.view(torch.float16).float(), q.float())
    assert torch.equal(dt[:, :m].t().contiguous().view(torch.int32), d.view(torch.int32))


@pytest.mark.parametrize("m,k", [(1, 4096), (7, 1280), (40, 2304)])
def test_norm_is_the_quantizer_of_its_y(m, k):
    """In f32, y is unrounded: the quants and scales are bit for bit the quantizer's of y."""
    ensure_built()
    x, r, w = make(m, k, "f32", seed=3)
    y = torch.empty((m, k), device="cuda")
    q, d = q8.rmsnorm_q8_1(x.cuda(), w.cuda(), residual=r.cuda(), y=y)
    q2, d2 = q8.quantize_q8_1(y)
    device_ok()
    assert torch.equal(q, q2) and torch.equal(d.view(torch.int32), d2.view(torch.int32))


def test_norm_strided_rows_and_in_place():
    """Rows of a wider buffer; the residual updated in place, or in x's own rows."""
    ensure_built()
    m, k = 9, 512
    for kind in ("f32", "bf16"):
        x, r, w = make(m, k, kind, seed=5)
        want_q, want_d = q8.rmsnorm_q8_1(x.cuda(), w.cuda(), residual=r.cuda())
        s_ref, _ = ref.rmsnorm(x, r, w, 1e-6)
        wide = torch.full((m, k + 64), 7.0, dtype=x.dtype, device="cuda")
        wide[:, 32:32 + k] = x.cuda()
        rr = torch.full((2 * m, k), 5.0, dtype=x.dtype, device="cuda")
        rr[::2] = r.cuda()
        q, d = q8.rmsnorm_q8_1(wide[:, 32:32 + k], w.cuda(), residual=rr[::2], residual_out=rr[::2])
        device_ok()
        assert torch.equal(q, want_q) and torch.equal(d, want_d)
        assert torch.equal(rr[::2].cpu(), s_ref) and bool((rr[1::2] == 5.0).all())
        q, d = q8.rmsnorm_q8_1(wide[:, 32:32 + k], w.cuda(), residual=r.cuda(), residual_out=wide[:, 32:32 + k])
        device_ok()
        assert torch.equal(q, want_q) and torch.equal(d, want_d)
        assert torch.equal(wide[:, 32:32 + k].cpu(), s_ref)
        assert bool((wide[:, :32] == 7.0).all()) and bool((wide[:, 32 + k:] == 7.0).all())


def test_norm_weight_types_and_none():
    ensure_built()
    m, k = 4, 1024
    x, _, _ = make(m, k, "bf16", residual=False)
    g = torch.Generator().manual_seed(9)
    for wt in (None, torch.float32, torch.float16, torch.bfloat16):
        w = None if wt is None else (1 + 0.2 * torch.randn(k, generator=g)).to(wt)
        _, y64 = ref.rmsnorm(x, None, w, 1e-6)
        q, d = q8.rmsnorm_q8_1(x.cuda(), None if w is None else w.cuda())
        device_ok()
        check_blocks(host(q).astype(np.float64), host(d).astype(np.float64), y64, k)


def test_norm_zero_tiny_and_nonfinite_rows():
    """A row of zeros gives zeros; tiny rows are scaled up as far as eps lets them; a row with a NaN
    or an infinity gives what the quantizers give for its y, and no other row changes."""
    ensure_built()
    m, k = 6, 256
    x, r, w = make(m, k, "f32", seed=7)
    clean_q, clean_d = q8.rmsnorm_q8_1(x.cuda(), w.cuda(), residual=r.cuda())
    x[1], r[1] = 0, 0
    x[2], r[2] = x[2] * 1e-30, 0
    x[3, 17] = float("nan")
    x[4, 200] = float("inf")
    y = torch.empty((m, k), device="cuda")
    q, d = q8.rmsnorm_q8_1(x.cuda(), w.cuda(), residual=r.cuda(), y=y)
    q2, d2 = q8.quantize_q8_1(y)
    device_ok()
    assert torch.equal(q, q2) and torch.equal(d.view(torch.int32), d2.view(torch.int32))
    assert not q[1].any() and not d[1].any() and not y[1].any()
    for i in (0, 5):
        assert torch.equal(q[i], clean_q[i]) and torch.equal(d[i], clean_d[i])
    _, y64 = ref.rmsnorm(x[2:3], r[2:3], w, 1e-6)
    check_blocks(host(q[2:3]).astype(np.float64), host(d[2:3]).astype(np.float64), y64, k)


@pytest.mark.parametrize("m,k", [(3, 1024), (700, 512), (2, 40960)])
def test_norm_alone(m, k):
    """The norm without quants is the quantizing norm's y, and updates the residual alike."""
    ensure_built()
    for kind in ("f32", "f16", "bf16"):
        x, r, w = make(m, k, kind, seed=13)
        x, r, w = x.cuda(), r.cuda(), w.cuda()
        y, s, s2 = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
        q8.rmsnorm_q8_1(x, w, residual=r, residual_out=s, y=y)
        out = torch.empty_like(x)
        assert q8.rmsnorm(x, w, residual=r, residual_out=s2, out=out) is out
        device_ok()
        assert torch.equal(out, y) and torch.equal(s, s2)


def test_norm_writes_only_its_outputs():
    ensure_built()
    m, k = 5, 768
    x, r, w = make(m, k, "f16")
    dev = torch.device("cuda")
    q = torch.full((m + 2, k), 99, dtype=torch.int8, device=dev)
    d = torch.full((m + 2, k // 32), 99.0, device=dev)
    q8.rmsnorm_q8_1(x.to(dev), w.to(dev), residual=r.to(dev), out=(q[1:m + 1], d[1:m + 1]))
    ldm = q8.q8act_mmq_ldm(m)
    qh = torch.full((m + 2, k), 9, dtype=torch.uint16, device=dev)
    dt = torch.full((k // 32, ldm), 99.0, device=dev)
    q8.rmsnorm_q8_1_mmq(x.to(dev), w.to(dev), residual=r.to(dev), out=(qh[1:m + 1], dt))
    device_ok()
    for buf, v in ((q, 99), (d, 99.0)):
        assert bool((buf[0] == v).all()) and bool((buf[m + 1] == v).all())
    assert bool((qh[0].int() == 9).all()) and bool((qh[m + 1].int() == 9).all())
    assert bool((dt[:, m:] == 99.0).all())          # columns beyond m are not written


def test_norm_feeds_the_products_on_its_stream():
    """norm -> GEMV and norm -> GEMM on a side stream equal the same calls made apart."""
    ensure_built()
    m, n, k = 4, 300, 512
    x, r, w = make(m, k, "bf16", seed=11)
    g = torch.Generator().manual_seed(1)
    wq = q8.quantize_q8_0((torch.randn((n, k), generator=g) * 0.02).cuda())
    x, r, w = x.cuda(), r.cuda(), w.cuda()
    q, d = q8.rmsnorm_q8_1(x, w, residual=r)
    qh, dt = q8.rmsnorm_q8_1_mmq(x, w, residual=r)
    y1, y2 = q8.gemv_q8_0(wq, q, d, n), q8.gemm_q8_0_preq(wq, qh, dt, n)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        big = torch.randn((4096, 4096), device="cuda")
        big = big @ big                                # the side stream is busy for a while
        xs = (x.float() + 0 * big[:m, :k]).to(x.dtype)   # and x comes from it
        a = q8.gemv_q8_0(wq, *q8.rmsnorm_q8_1(xs, w, residual=r), n)
        b = q8.gemm_q8_0_preq(wq, *q8.rmsnorm_q8_1_mmq(xs, w, residual=r), n)
    side.synchronize()
    device_ok()
    assert torch.equal(a, y1) and torch.equal(b, y2)
