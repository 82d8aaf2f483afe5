"""GB300 (sm_103a) Q8_0 weight x q8_1 activation block-quantized matmul, and what stands next to it
in a decoder: the norm that feeds it, MXFP4 products, log probabilities of logits.

The compute lives in libq8act.so (hand-written CUDA kernels behind the C ABI of
include/q8act.h).  This package is its Python face:

  * the raw ABI under the C names (``q8act_quantize_q8_1``, ``q8act_gemv_q8_0``, ...), which
    take torch tensors or integer device addresses and return the C return code;
  * torch conveniences (``quantize_q8_1``, ``gemv_q8_0``, ``gemm_q8_0``, ...) that allocate
    outputs with torch on the input's device, call the ABI on torch's current stream and
    raise ``Q8ActError`` on a non-zero return code.

There is no CPU or PyTorch fallback: without the built library every call raises.
"""
from __future__ import annotations

from ._lib import (  # noqa: F401  (re-exported ABI)
    EXPORTED, LIB_PATH, Q8ACT_ERR_ALIGN, Q8ACT_ERR_CUDA_BASE, Q8ACT_ERR_DEVICE, Q8ACT_ERR_DIMS,
    Q8ACT_ERR_NULL, Q8ACT_ERR_TIMEOUT, Q8ACT_ERR_WORKSPACE, Q8ACT_GEMV_MAX_M, Q8ACT_MAX_K,
    Q8ACT_NOALLOC_WS_BYTES, Q8ACT_GEMM_SPLIT_BYTES, Q8ACT_OK, Q8ActError, check, lib, q8act_debug_gemm_block_dots, q8act_debug_gemv_block_dots,
    q8act_dequant_q8_0_f16, q8act_device_status, q8act_gemm_q8_0, q8act_gemm_q8_0_preq,
    q8act_gemm_q8_0_noalloc, q8act_gemm_workspace_bytes, q8act_gemv_q8_0, q8act_mmq_ldm, q8act_quantize_q8_0,
    q8act_quantize_q8_1, q8act_quantize_q8_1_mmq, q8act_strerror, q8act_version, strerror,
    q8act_repack_q8_0, q8act_repack_ldn, q8act_gemm_q8_0_repacked, q8act_debug_gemm_repacked_block_dots,
    q8act_gemv_q8_0_group, Q8ACT_GEMV_MAX_GROUP, q8act_quantize_q4_0, q8act_dequant_q4_0_f16,
    q8act_gemv_q4_0, q8act_debug_gemv_q4_0_block_dots, q8act_gemv_workspace_bytes, q8act_gemv_q8_0_f32,
    q8act_debug_wait_timeout, Q8ACT_ERR_DRAIN_TIMEOUT, Q8ACT_GEMV_KQ_MAX_M,
    q8act_dequant_q6_k_f16, q8act_dequant_q4_k_f16, q8act_dequant_q5_k_f16,
    q8act_gemv_q6_k, q8act_gemv_q4_k, q8act_gemv_q5_k,
    q8act_debug_gemv_q6_k_block_dots, q8act_debug_gemv_q4_k_block_dots, q8act_debug_gemv_q5_k_block_dots,
    Q8ACT_ERR_TYPE, Q8ACT_F32, Q8ACT_F16, Q8ACT_BF16, Q8ACT_MAX_TOP, q8act_rmsnorm_q8_1, q8act_rmsnorm_q8_1_mmq,
    q8act_mxfp4_scale_bytes, q8act_quantize_mxfp4, q8act_dequant_mxfp4, q8act_tile_mxfp4_scales,
    q8act_gemm_mxfp4_workspace_bytes, q8act_gemm_mxfp4, q8act_gemm_mxfp4_preq,
    q8act_debug_gemm_mxfp4_plan, q8act_logprobs)

QK = 32
Q8_0_BYTES = 34
Q4_0_BYTES = 18


def row_bytes(k: int) -> int:
    """Bytes of one Q8_0 row of k values (k/32 blocks of 34 bytes)."""
    return k // QK * Q8_0_BYTES


def quantize_q8_0(w):
    """f32 [n, k] CUDA tensor -> Q8_0 bytes, uint8 [n, k/32*34]."""
    import torch
    n, k = w.shape
    out = torch.empty((n, row_bytes(k)), dtype=torch.uint8, device=w.device)
    check(q8act_quantize_q8_0(w, out, n, k), "q8act_quantize_q8_0")
    return out


def quantize_q8_1(x):
    """f32 [m, k] -> (xq int8 [m, k], xd f32 [m, k/32])."""
    import torch
    m, k = x.shape
    xq = torch.empty((m, k), dtype=torch.int8, device=x.device)
    xd = torch.empty((m, k // QK), dtype=torch.float32, device=x.device)
    check(q8act_quantize_q8_1(x, xq, xd, m, k), "q8act_quantize_q8_1")
    return xq, xd


def quantize_q8_1_mmq(x):
    """f32 [m, k] -> (xqh uint16 [m, k] binary16 quants, xdt f32 [k/32, ldm] scales)."""
    import torch
    m, k = x.shape
    xqh = torch.empty((m, k), dtype=torch.uint16, device=x.device)
    xdt = torch.empty((k // QK, q8act_mmq_ldm(m)), dtype=torch.float32, device=x.device)
    check(q8act_quantize_q8_1_mmq(x, xqh, xdt, m, k), "q8act_quantize_q8_1_mmq")
    return xqh, xdt


def gemv_q8_0(w, xq, xd, n: int, out=None):
    """Decode GEMV: Q8_0 bytes w (n rows), q8_1 activation (xq, xd) of m <= Q8ACT_GEMV_MAX_M (15) tokens."""
    import torch
    m, k = xq.shape
    y = out if out is not None else torch.empty((m, n), dtype=torch.float32, device=xq.device)
    check(q8act_gemv_q8_0(w, xq, xd, y, m, n, k), "q8act_gemv_q8_0")
    return y


def gemv_q8_0_group(ws, xq, xd, ns, outs=None):
    """Grouped decode GEMV: weight matrices ws (Q8_0 bytes of ns[i] rows each) sharing the
    q8_1 activation (xq, xd) of m tokens, one launch; returns the list of outputs."""
    import torch
    m, k = xq.shape
    ys = outs if outs is not None else [torch.empty((m, n), dtype=torch.float32, device=xq.device) for n in ns]
    check(q8act_gemv_q8_0_group(ws, ys, ns, xq, xd, m, k), "q8act_gemv_q8_0_group")
    return ys


def gemm_workspace(m: int, k: int, device):
    import torch
    nbytes = q8act_gemm_workspace_bytes(m, k)
    if nbytes == 0:
        raise Q8ActError(Q8ACT_ERR_DIMS, "q8act_gemm_workspace_bytes")
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def gemm_q8_0(w, x, n: int, ws=None, out=None):
    """Prefill GEMM with the q8_1 quantization of x fused into the call."""
    import torch
    m, k = x.shape
    if ws is None:
        ws = gemm_workspace(m, k, x.device)
    y = out if out is not None else torch.empty((m, n), dtype=torch.float32, device=x.device)
    check(q8act_gemm_q8_0(w, x, y, m, n, k, ws, ws.numel()), "q8act_gemm_q8_0")
    return y


def gemm_q8_0_preq(w, xqh, xdt, n: int, out=None):
    """Prefill GEMM on an activation already in the MMQ layout (quantize_q8_1_mmq)."""
    import torch
    m, k = xqh.shape
    y = out if out is not None else torch.empty((m, n), dtype=torch.float32, device=xqh.device)
    check(q8act_gemm_q8_0_preq(w, xqh, xdt, y, m, n, k), "q8act_gemm_q8_0_preq")
    return y


def repack_q8_0(w, n: int, k: int):
    """Load-time repack of Q8_0 bytes for the tensor-core GEMM: (wq16 float16 [n, k] holding
    the exact quants, wdt float32 [k/32, q8act_repack_ldn(n)] holding the block scales)."""
    import torch
    wq16 = torch.empty((n, k), dtype=torch.float16, device=w.device)
    wdt = torch.zeros((k // QK, q8act_repack_ldn(n)), dtype=torch.float32, device=w.device)
    check(q8act_repack_q8_0(w, wq16, wdt, n, k), "q8act_repack_q8_0")
    return wq16, wdt


def gemm_q8_0_repacked(wq16, wdt, x, ws=None, out=None):
    """Prefill GEMM (q8_1 quantization fused) on repacked weights (repack_q8_0)."""
    import torch
    m, k = x.shape
    n = wq16.shape[0]
    if ws is None:
        ws = gemm_workspace(m, k, x.device)
    y = out if out is not None else torch.empty((m, n), dtype=torch.float32, device=x.device)
    check(q8act_gemm_q8_0_repacked(wq16, wdt, x, y, m, n, k, ws, ws.numel()), "q8act_gemm_q8_0_repacked")
    return y


def dequant_q8_0_f16(w, n: int, k: int, out=None):
    """Q8_0 bytes -> row-major float16 [n, k]."""
    import torch
    w16 = out if out is not None else torch.empty((n, k), dtype=torch.float16, device=w.device)
    check(q8act_dequant_q8_0_f16(w, w16, n, k), "q8act_dequant_q8_0_f16")
    return w16


def device_status(stream=None) -> None:
    """Synchronize and raise if a kernel recorded a pipeline timeout since the last check."""
    check(q8act_device_status(stream), "q8act_device_status")


def row_bytes_q4_0(k: int) -> int:
    """Bytes of one Q4_0 row of k values (k/32 blocks of 18 bytes)."""
    return k // QK * Q4_0_BYTES


def quantize_q4_0(w):
    """f32 [n, k] CUDA tensor -> Q4_0 bytes, uint8 [n, k/32*18] (data preparation)."""
    import torch
    n, k = w.shape
    out = torch.empty((n, row_bytes_q4_0(k)), dtype=torch.uint8, device=w.device)
    check(q8act_quantize_q4_0(w, out, n, k), "q8act_quantize_q4_0")
    return out


def dequant_q4_0_f16(w, n: int, k: int, out=None):
    """Q4_0 bytes -> row-major float16 [n, k]."""
    import torch
    w16 = out if out is not None else torch.empty((n, k), dtype=torch.float16, device=w.device)
    check(q8act_dequant_q4_0_f16(w, w16, n, k), "q8act_dequant_q4_0_f16")
    return w16


def gemv_q4_0(w, xq, xd, n: int, out=None):
    """Q4_0 weights x pre-quantized q8_1 activation: y f32 [m, n] (1 <= m <= 15)."""
    import torch
    m, k = xq.shape
    y = out if out is not None else torch.empty((m, n), dtype=torch.float32, device=xq.device)
    check(q8act_gemv_q4_0(w, xq, xd, y, m, n, k), "q8act_gemv_q4_0")
    return y


def gemv_workspace(m: int, k: int, device):
    """A workspace for the fused GEMV (q8act_gemv_q8_0_f32)."""
    import torch
    nbytes = q8act_gemv_workspace_bytes(m, k)
    if nbytes == 0:
        raise Q8ActError(Q8ACT_ERR_DIMS, "q8act_gemv_workspace_bytes")
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def gemv_q8_0_f32(w, x, n: int, ws=None, out=None):
    """Decode GEMV with the q8_1 quantization fused: f32 x [m, k] -> y f32 [m, n]."""
    import torch
    m, k = x.shape
    if ws is None:
        ws = gemv_workspace(m, k, x.device)
    y = out if out is not None else torch.empty((m, n), dtype=torch.float32, device=x.device)
    check(q8act_gemv_q8_0_f32(w, x, y, m, n, k, ws, ws.numel()), "q8act_gemv_q8_0_f32")
    return y


KQ_BYTES = {"q6_k": 210, "q4_k": 144, "q5_k": 176}   # bytes per 256-weight superblock


def dequant_kq_f16(fmt: str, w, n: int, k: int, out=None):
    """K-quant superblocks (fmt "q6_k", "q4_k" or "q5_k") -> row-major float16 [n, k]."""
    import torch
    w16 = out if out is not None else torch.empty((n, k), dtype=torch.float16, device=w.device)
    fn = {"q6_k": q8act_dequant_q6_k_f16, "q4_k": q8act_dequant_q4_k_f16, "q5_k": q8act_dequant_q5_k_f16}[fmt]
    check(fn(w, w16, n, k), f"q8act_dequant_{fmt}_f16")
    return w16


def gemv_kq(fmt: str, w, xq, xd, n: int, out=None):
    """Decode GEMV over K-quant weights (n rows) with the q8_1 activation of m <= 8 tokens."""
    import torch
    m, k = xq.shape
    y = out if out is not None else torch.empty((m, n), dtype=torch.float32, device=xq.device)
    fn = {"q6_k": q8act_gemv_q6_k, "q4_k": q8act_gemv_q4_k, "q5_k": q8act_gemv_q5_k}[fmt]
    check(fn(w, xq, xd, y, m, n, k), f"q8act_gemv_{fmt}")
    return y


# The calls below take several element types, row strides and caller's buffers; they are made once
# per layer and token, so their checks are kept to a few attribute reads (a microsecond or two a
# call) and the addresses go straight to the C ABI.
_TYPES: dict = {}
_torch = None
_current = None      # the current CUDA device's index, as a call
_stream = None       # torch's current stream on a device, as an address


def _load_torch():
    global _torch, _current, _stream
    import torch
    if torch.cuda.is_available():
        _current, _stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
    else:
        _current = lambda: -2                    # noqa: E731  no tensor's
    _TYPES.update({torch.float32: Q8ACT_F32, torch.float16: Q8ACT_F16, torch.bfloat16: Q8ACT_BF16})
    _torch = torch
    return torch


def _type(t, what: str) -> int:
    """The element type code of a tensor."""
    code = _TYPES.get(t.dtype)
    if code is None:
        raise Q8ActError(Q8ACT_ERR_TYPE, f"{what}: {t.dtype}")
    return code


def _elsewhere(t, what: str, dev: int):
    """The kernels run on the current device and its current stream: a tensor of another GPU would be a
    foreign address there, unordered with the work that made it."""
    return Q8ActError(Q8ACT_ERR_DEVICE, f"{what}: not on the current CUDA device (cuda:{dev})" if t.is_cuda
                      else f"{what}: not a CUDA tensor")


def _rows(t, what: str, dev: int) -> int:
    """Row stride in elements of a [rows, columns] tensor on device dev whose columns are adjacent."""
    if t.get_device() != dev:
        raise _elsewhere(t, what, dev)
    shape = t.shape
    if len(shape) == 2 and shape[0] > 0:
        if t.is_contiguous():
            return shape[1]
        if t.stride(1) == 1 or shape[1] <= 1:
            return t.stride(0)
    raise Q8ActError(Q8ACT_ERR_DIMS, f"{what}: one row at least, with adjacent columns")


def _given(t, shape, dtype, what: str, dev: int):
    """The address of a caller's buffer on device dev: the kernels write or read exactly `shape`."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    if t.get_device() != dev:
        raise _elsewhere(t, what, dev)
    if t.dtype is not dtype:
        raise Q8ActError(Q8ACT_ERR_TYPE, f"{what}: {t.dtype}")
    raise Q8ActError(Q8ACT_ERR_DIMS, f"{what}: contiguous {tuple(shape)}")


def _rmsnorm(mmq, x, weight, eps, residual, residual_out, y, out, quants=True):
    torch = _torch or _load_torch()
    dev = _current()
    ldx, code = _rows(x, "x", dev), _type(x, "x")
    m, k = shape = x.shape
    dtype = x.dtype
    pr = pro = pw = py = None
    ldr = ldro = wtype = 0
    if residual is not None:
        ldr, pr = _rows(residual, "residual", dev), residual.data_ptr()
        if residual.dtype is not dtype or residual.shape != shape:
            raise Q8ActError(Q8ACT_ERR_TYPE, "residual: x's type and shape")
    if residual_out is not None:
        ldro, pro = _rows(residual_out, "residual_out", dev), residual_out.data_ptr()
        if residual_out.dtype is not dtype or residual_out.shape != shape:
            raise Q8ActError(Q8ACT_ERR_TYPE, "residual_out: x's type and shape")
    if weight is not None:
        wtype, pw = _type(weight, "weight"), _given(weight, (k,), weight.dtype, "weight", dev)
    if y is not None:
        py = _given(y, shape, dtype, "y", dev)
    qtype, dshape = (torch.uint16, (k // QK, (m + 3) // 4 * 4)) if mmq else (torch.int8, (m, k // QK))
    if not quants:
        q = d = pq = pd = None
    else:
        if out is None:
            out = (torch.empty(shape, dtype=qtype, device=x.device),
                   torch.empty(dshape, dtype=torch.float32, device=x.device))
        q, d = out
        pq, pd = _given(q, shape, qtype, "quants", dev), _given(d, dshape, torch.float32, "scales", dev)
    L = lib()
    fn = L.q8act_rmsnorm_q8_1_mmq if mmq else L.q8act_rmsnorm_q8_1
    rc = fn(x.data_ptr(), ldx, pr, ldr, pw, wtype, eps, pro, ldro, py, pq, pd, m, k, code, _stream(dev))
    if rc:
        raise Q8ActError(rc, "q8act_rmsnorm_q8_1_mmq" if mmq else "q8act_rmsnorm_q8_1")
    return q, d


def rmsnorm_q8_1(x, weight=None, eps: float = 1e-6, residual=None, residual_out=None, y=None, out=None):
    """Residual addition, RMS norm and q8_1 quantization in one call: s = x + residual,
    y = s * rsqrt(mean(s^2) + eps) * weight -> (xq int8 [m, k], xd f32 [m, k/32]) for the GEMVs.
    x, residual: float32, float16 or bfloat16 rows (any row stride whose rows stay 16-byte
    aligned); residual_out (may be residual or x itself) receives s, y the normed values, both
    in x's type."""
    return _rmsnorm(False, x, weight, eps, residual, residual_out, y, out)


def rmsnorm_q8_1_mmq(x, weight=None, eps: float = 1e-6, residual=None, residual_out=None, y=None, out=None):
    """rmsnorm_q8_1 with the GEMM's activation layout: (xqh uint16 [m, k], xdt f32 [k/32, ldm])."""
    return _rmsnorm(True, x, weight, eps, residual, residual_out, y, out)


def rmsnorm(x, weight=None, eps: float = 1e-6, residual=None, residual_out=None, out=None):
    """The norm alone: y in x's type (what rmsnorm_q8_1 gives as y), for a consumer that is not
    quantized to q8_1, such as an MXFP4 product."""
    torch = _torch or _load_torch()
    dev = _current()
    _rows(x, "x", dev)
    y = out if out is not None else torch.empty(x.shape, dtype=x.dtype, device=x.device)
    _rmsnorm(False, x, weight, eps, residual, residual_out, y, None, quants=False)
    return y


def _mxfp4_scales(rows: int, k: int):
    """Shape of a tiled scale array (q8act_mxfp4_scale_bytes)."""
    if rows < 1 or k < 1 or k % 256 or k > Q8ACT_MAX_K:
        raise Q8ActError(Q8ACT_ERR_DIMS, f"MXFP4 matrix of {rows} x {k}")
    return ((rows + 127) // 128 * (k // 128) * 512,)


def quantize_mxfp4(x, out=None):
    """float32, float16 or bfloat16 [m, k] -> MXFP4 (codes uint8 [m, k/2], tiled scales uint8)."""
    torch = _torch or _load_torch()
    dev = _current()
    ldx, code = _rows(x, "x", dev), _type(x, "x")
    m, k = x.shape
    u8, nsc = torch.uint8, _mxfp4_scales(m, k)
    if out is None:
        out = (torch.empty((m, k // 2), dtype=u8, device=x.device), torch.empty(nsc, dtype=u8, device=x.device))
    codes, scales = out
    rc = lib().q8act_quantize_mxfp4(x.data_ptr(), ldx, code, _given(codes, (m, k // 2), u8, "codes", dev),
                                    _given(scales, nsc, u8, "scales", dev), m, k, _stream(dev))
    if rc:
        raise Q8ActError(rc, "q8act_quantize_mxfp4")
    return codes, scales


def dequant_mxfp4(codes, scales, dtype=None, out=None):
    """MXFP4 (codes, tiled scales) -> values [m, k] in dtype (default float16) or out's type."""
    torch = _torch or _load_torch()
    dev = _current()
    m, half = codes.shape
    k, u8 = 2 * half, torch.uint8
    pc, ps = _given(codes, (m, half), u8, "codes", dev), _given(scales, _mxfp4_scales(m, k), u8, "scales", dev)
    if out is None:
        out = torch.empty((m, k), dtype=dtype or torch.float16, device=codes.device)
    code = _type(out, "out")
    rc = lib().q8act_dequant_mxfp4(pc, ps, _given(out, (m, k), out.dtype, "out", dev), code, m, k, _stream(dev))
    if rc:
        raise Q8ActError(rc, "q8act_dequant_mxfp4")
    return out


def tile_mxfp4_scales(scales):
    """Row-major e8m0 bytes [m, k/32] -> the tiled scales that the MXFP4 calls take."""
    torch = _torch or _load_torch()
    dev = _current()
    m, kb = scales.shape
    ps = _given(scales, (m, kb), torch.uint8, "scales", dev)
    tiled = torch.empty(_mxfp4_scales(m, kb * QK), dtype=torch.uint8, device=scales.device)
    rc = lib().q8act_tile_mxfp4_scales(ps, tiled.data_ptr(), m, kb * QK, _stream(dev))
    if rc:
        raise Q8ActError(rc, "q8act_tile_mxfp4_scales")
    return tiled


def gemm_mxfp4_workspace(m: int, k: int, device):
    """A workspace for gemm_mxfp4 (the quantized activation)."""
    import torch
    nbytes = q8act_gemm_mxfp4_workspace_bytes(m, k)
    if nbytes == 0:
        raise Q8ActError(Q8ACT_ERR_DIMS, "q8act_gemm_mxfp4_workspace_bytes")
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def gemm_mxfp4(w, wscales, x, ws=None, dtype=None, out=None):
    """x [m, k] (float32, float16, bfloat16; quantized to MXFP4 in the call) times MXFP4 weights
    (codes w [n, k/2], tiled scales): y [m, n] in dtype (default float32) or out's type."""
    torch = _torch or _load_torch()
    dev = _current()
    n, half = w.shape
    k, u8 = 2 * half, torch.uint8
    pw, psc = _given(w, (n, half), u8, "w", dev), _given(wscales, _mxfp4_scales(n, k), u8, "wscales", dev)
    ldx, code = _rows(x, "x", dev), _type(x, "x")
    m = x.shape[0]
    if x.shape[1] != k:
        raise Q8ActError(Q8ACT_ERR_DIMS, f"x: {x.shape[1]} columns for weights of {k}")
    if ws is None:
        ws = gemm_mxfp4_workspace(m, k, x.device)
    elif ws.get_device() != dev:
        raise _elsewhere(ws, "ws", dev)
    elif not (ws.dtype is u8 and ws.is_contiguous()):
        raise Q8ActError(Q8ACT_ERR_WORKSPACE, "ws: contiguous uint8")
    if out is None:
        out = torch.empty((m, n), dtype=dtype or torch.float32, device=x.device)
    ycode = _type(out, "out")
    rc = lib().q8act_gemm_mxfp4(pw, psc, x.data_ptr(), ldx, code, _given(out, (m, n), out.dtype, "out", dev), ycode,
                                m, n, k, ws.data_ptr(), ws.numel(), _stream(dev))
    if rc:
        raise Q8ActError(rc, "q8act_gemm_mxfp4")
    return out


def gemm_mxfp4_preq(w, wscales, xq, xscales, dtype=None, out=None):
    """The product on an activation already in MXFP4 (quantize_mxfp4)."""
    torch = _torch or _load_torch()
    dev = _current()
    n, half = w.shape
    k, u8, m = 2 * half, torch.uint8, xq.shape[0]
    pw, psc = _given(w, (n, half), u8, "w", dev), _given(wscales, _mxfp4_scales(n, k), u8, "wscales", dev)
    px, pxs = _given(xq, (m, half), u8, "xq", dev), _given(xscales, _mxfp4_scales(m, k), u8, "xscales", dev)
    if out is None:
        out = torch.empty((m, n), dtype=dtype or torch.float32, device=xq.device)
    ycode = _type(out, "out")
    rc = lib().q8act_gemm_mxfp4_preq(pw, psc, px, pxs, _given(out, (m, n), out.dtype, "out", dev), ycode, m, n, k,
                                     _stream(dev))
    if rc:
        raise Q8ActError(rc, "q8act_gemm_mxfp4_preq")
    return out


def logprobs(logits, tokens=None, top: int = 0, out=None):
    """For each row of logits [m, v] (float32, float16, bfloat16; -inf = masked): the log
    probability of tokens[row] (int32; negative: none, 0), the entropy, and the `top` most likely
    ids (int32 [m, top], equal logits by the lower id, -1 beyond the unmasked ones) with their
    log probabilities.  Returns (logprob or None, entropy, ids, top_logprobs)."""
    torch = _torch or _load_torch()
    dev = _current()
    ld, code = _rows(logits, "logits", dev), _type(logits, "logits")
    m, v = logits.shape
    f32, i32 = torch.float32, torch.int32
    ptok = plp = pids = ptlp = None
    if out is None:
        at, n = logits.device, max(top, 0)
        out = (torch.empty(m, dtype=f32, device=at) if tokens is not None else None,
               torch.empty(m, dtype=f32, device=at), torch.empty((m, n), dtype=i32, device=at),
               torch.empty((m, n), dtype=f32, device=at))
    lp, ent, ids, tlp = out
    if tokens is not None:
        ptok, plp = _given(tokens, (m,), i32, "tokens", dev), _given(lp, (m,), f32, "logprob", dev)
    if top > 0:
        pids, ptlp = _given(ids, (m, top), i32, "ids", dev), _given(tlp, (m, top), f32, "top_logprobs", dev)
    rc = lib().q8act_logprobs(logits.data_ptr(), ld, code, ptok, plp, _given(ent, (m,), f32, "entropy", dev), pids, ptlp,
                              m, v, top, _stream(dev))
    if rc:
        raise Q8ActError(rc, "q8act_logprobs")
    return lp, ent, ids, tlp
