"""Plain 64-bit forms of the norm, the MXFP4 format and product, and the log probabilities: what
their GPU tests compare with.  numpy and torch on the CPU; nothing of the library's code."""
import numpy as np
import torch

QK = 32
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -24                       # half a unit in the last place of f32
HALF_ULP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def f64(t):
    return t.detach().cpu().double().numpy()


def rmsnorm(x, r, w, eps):
    """x, r, w CPU tensors -> (residual sum as the type of x, y in 64 bits)."""
    s = x.float() if r is None else x.float() + r.float()
    s64 = f64(s)
    y = s64 / np.sqrt((s64 * s64).mean(1, keepdims=True) + np.float64(np.float32(eps)))
    return s.to(x.dtype), y if w is None else y * f64(w)


def mxfp4_quantize(x):
    """f64 [m][k] -> (scale bytes [m][k/32] uint8, codes [m][k] uint8 in 0..15)."""
    m, k = x.shape
    b = x.reshape(m, k // QK, QK)
    with np.errstate(invalid="ignore"):
        amax = np.abs(b).max(-1)
    bad = ~np.isfinite(amax)
    safe = np.where(bad, 0.0, amax)
    e = np.maximum(np.frexp(safe)[1] - 3, -127)          # floor(log2 amax) - 2
    e = np.where(safe == 0, -127, e)
    v = np.where(bad[..., None], 0.0, b) / np.exp2(e.astype(np.float64))[..., None]
    a = np.abs(v)
    d = np.abs(a[..., None] - E2M1)
    near = d == d.min(-1, keepdims=True)
    # of two equally near values, the one with the even code
    score = near * (2 + (np.arange(8) % 2 == 0))
    code = score.argmax(-1).astype(np.uint8)
    code |= (np.signbit(v).astype(np.uint8) << 3)
    byte = np.where(bad, 255, e + 127).astype(np.uint8)
    return byte, code.reshape(m, k)


def mxfp4_values(byte, code):
    v = E2M1[code & 7] * np.where(code & 8, -1.0, 1.0)
    s = np.where(byte == 255, np.nan, np.exp2(byte.astype(np.float64) - 127))
    return v * np.repeat(s, QK, 1)


def pack_codes(code):
    return (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8)


def tile_scales(byte, fill=0):
    m, kb = byte.shape
    out = np.full((m + 127) // 128 * (kb // 4) * 512, fill, np.uint8)
    r, b = np.meshgrid(np.arange(m), np.arange(kb), indexing="ij")
    out[((r // 128) * (kb // 4) + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4] = byte
    return out


def logprobs(x, tokens, top):
    """f64 [m][v] -> (logprob, entropy, ids, top log probabilities)."""
    m, v = x.shape
    lp, ent = np.zeros(m), np.zeros(m)
    ids, tlp = np.full((m, top), -1, np.int32), np.full((m, top), -np.inf)
    for i, row in enumerate(x):
        if np.isnan(row).any() or (row == np.inf).any():
            lp[i] = ent[i] = np.nan
            tlp[i] = np.nan
        else:
            mx = row.max()
            p = row - mx - np.log(np.exp(row - mx).sum()) if mx > -np.inf else row
            live = p > -np.inf
            ent[i] = -(p[live] * np.exp(p[live])).sum()
            order = np.lexsort((np.arange(v), -row))
            order = order[live[order]][:top]
            ids[i, :len(order)], tlp[i, :len(order)] = order, p[order]
            if tokens is not None and 0 <= tokens[i] < v:
                lp[i] = p[tokens[i]]
        if tokens is not None:
            lp[i] = 0.0 if tokens[i] < 0 else np.nan if tokens[i] >= v else lp[i]
    return lp, ent, ids, tlp
