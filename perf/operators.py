"""Operators around the block-quantized products of a decoder, and how they are measured.

Four operators, as a serving step meets them:

  norm      residual addition + root-mean-square norm + q8_1 quantization, in the two layouts
            that the products read ("q8_1": int8 quants and row-major scales for the GEMVs,
            "mmq": binary16 quants and block-major scales for the GEMM)
  quantize  MXFP4 quantization (blocks of 32, e2m1 codes, e8m0 scales) and back to values
  product   f32 / f16 / bf16 activation, quantized to MXFP4, times MXFP4 weights
  logprobs  log probability of a given token, entropy and the top alternatives of logits rows

`own` selects the framework's kernels; otherwise each operator is computed from elementary
torch operations in 32 bits.
"""
import math

import numpy as np
import torch

own = False

QK = 32
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-6


# ---------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------
def listed():
    return [
        # one token between two decode GEMVs: latency
        dict(name="norm 1x4096 f32 q8_1", op="norm", m=1, k=4096, type="f32", residual=True, layout="q8_1"),
        # a prefill chunk in front of the GEMM
        dict(name="norm 512x4096 bf16 mmq", op="norm", m=512, k=4096, type="bf16", residual=True, layout="mmq"),
        # the largest chunk, wide model, the first norm (no residual yet), ragged
        dict(name="norm 4093x8192 f16 mmq", op="norm", m=4093, k=8192, type="f16", residual=False, layout="mmq"),
        # a few speculative tokens quantized and mirrored
        dict(name="quantize 7x4096 f32", op="quantize", m=7, k=4096, type="f32"),
        # a weight matrix at load time
        dict(name="quantize 20480x4096 bf16", op="quantize", m=20480, k=4096, type="bf16"),
        # decode: one token, one square projection
        dict(name="product 1x4096x4096 f32", op="product", m=1, n=4096, k=4096, type="f32", out="f32"),
        # speculative verify through the output head
        dict(name="product 5x64448x4096 f32", op="product", m=5, n=64448, k=4096, type="f32", out="f32"),
        # a ragged batch of sequences on a small projection
        dict(name="product 131x4096x1280 f16", op="product", m=131, n=4096, k=1280, type="f16", out="f16"),
        # a prefill chunk through the widest projection
        dict(name="product 512x20480x4096 bf16", op="product", m=512, n=20480, k=4096, type="bf16", out="bf16"),
        # the largest prefill
        dict(name="product 4095x20480x8192 bf16", op="product", m=4095, n=20480, k=8192, type="bf16", out="bf16"),
        # one decoded token with 20 alternatives
        dict(name="logprobs 1x64448 f32", op="logprobs", m=1, v=64448, type="f32", top=20, masked=False),
        # scoring a prompt under a constrained vocabulary
        dict(name="logprobs 509x128896 bf16", op="logprobs", m=509, v=128896, type="bf16", top=8, masked=True),
    ]


def _log(rng, lo, hi):
    while True:
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        if lo <= v <= hi and v != 3072:
            return v


def _k(rng, hi):
    return 256 * next(j for j in iter(lambda: _log(rng, 1, hi // 256), None) if j != 12)


def draw(rng):
    op = rng.choice(("norm", "quantize", "product", "logprobs"))
    kind = rng.choice(tuple(TYPES))
    if op == "norm":
        return dict(op=op, m=_log(rng, 1, 4093), k=_k(rng, 8192), type=kind, residual=rng.random() < 0.7,
                    layout=rng.choice(("q8_1", "mmq")))
    if op == "quantize":
        return dict(op=op, m=_log(rng, 1, 5120), k=_k(rng, 8192), type=kind)
    if op == "product":
        while True:
            m, n, k = _log(rng, 1, 4095), _log(rng, 64, 64448), _k(rng, 8192)
            if m * n <= 4095 * 20480 and m * n * k <= 4095 * 20480 * 8192 and n * k <= 20480 * 8192:
                return dict(op=op, m=m, n=n, k=k, type=kind, out=rng.choice(tuple(TYPES)))
    return dict(op=op, m=_log(rng, 1, 509), v=_log(rng, 1000, 128896), type=kind, top=rng.choice((1, 5, 8, 20, 32)),
                masked=rng.random() < 0.4)


# ---------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------
def _scale_bytes(rows, k):
    """Bytes of a tiled e8m0 scale array: 512 for each 128 rows x 128 values."""
    return -(-rows // 128) * (k // 128) * 512


def _tile(b):
    """Row-major scale bytes [rows][k/32] to tiles [rows/128][k/128][32][4][4]: the byte of row r and
    block b stands at (r / 128, b / 4, r % 32, r % 128 / 32, b % 4)."""
    rows, kb = b.shape
    full = torch.zeros((-(-rows // 128) * 128, kb), dtype=torch.uint8, device=b.device)
    full[:rows] = b
    return full.view(-1, 4, 32, kb // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _untile(t, rows, kb):
    return t.view(-1, kb // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, kb)[:rows]


def _pow2(e):
    """2^e in f32, e clamped to the normal exponents (only blocks of zeros lie below them here)."""
    return ((e.clamp(-126, 127) + 127).int() << 23).view(torch.float32)


def _mx(x):
    """f32 [rows][k] -> (codes' magnitudes 0..7, exponents E) of its MXFP4 blocks."""
    b = x.view(x.shape[0], -1, QK)
    amax = b.abs().amax(-1)
    e = (torch.frexp(amax).exponent - 3).clamp(-127, 127)     # floor(log2 amax) - 2
    e = torch.where(amax == 0, torch.full_like(e, -127), e)
    a = b.abs() * _pow2(-e).unsqueeze(-1)
    # round to the nearest of 0 0.5 1 1.5 2 3 4 6, ties to the even code
    c = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return c, e


def _magnitudes(device):
    return torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=device)


def _mx_values(x):
    """f32 [rows][k] -> the f32 values that its MXFP4 form stands for."""
    c, e = _mx(x)
    v = _magnitudes(x.device)[c.int()].copysign(x.view(c.shape))
    return (v * _pow2(e).unsqueeze(-1)).view(x.shape)


def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 16 + salt)
    return g


def _randn(shape, g):
    return torch.randn(shape, generator=g, device="cuda")


def _hidden(m, k, g):
    """Hidden states: unit normal, one value in a hundred 20 times larger."""
    x = _randn((m, k), g)
    return torch.where(torch.rand((m, k), generator=g, device="cuda") < 0.01, 20 * x, x)


def prepare(case, seed):
    op, m = case["op"], case["m"]
    t = TYPES[case["type"]]
    s = dict(case)
    if op == "norm":
        k = case["k"]
        s["x"] = _hidden(m, k, _gen(seed, 1)).to(t)
        s["r"] = (4 * _randn((m, k), _gen(seed, 2))).to(t) if case["residual"] else None
        s["w"] = (1 + 0.1 * _randn((k,), _gen(seed, 3))).to(t)
        s["r_out"] = torch.empty_like(s["x"]) if case["residual"] else None
        if case["layout"] == "q8_1":
            s["q"] = torch.empty((m, k), dtype=torch.int8, device="cuda")
            s["d"] = torch.empty((m, k // QK), device="cuda")
            s["values"] = torch.empty((m, k // QK, QK), dtype=torch.float16, device="cuda")
        else:
            s["q"] = torch.empty((m, k), dtype=torch.uint16, device="cuda")
            s["d"] = torch.empty((k // QK, -(-m // 4) * 4), device="cuda")
    elif op == "quantize":
        k = case["k"]
        s["x"] = _randn((m, k), _gen(seed, 1)).mul_(0.02).to(t)
        s["codes"] = torch.empty((m, k // 2), dtype=torch.uint8, device="cuda")
        s["scales"] = torch.empty(_scale_bytes(m, k), dtype=torch.uint8, device="cuda")
        s["values"] = torch.empty((m, k), dtype=torch.bfloat16, device="cuda")
    elif op == "product":
        n, k = case["n"], case["k"]
        s["w"] = torch.empty((n, k // 2), dtype=torch.uint8, device="cuda")
        bytes_ = torch.empty((n, k // QK), dtype=torch.uint8, device="cuda")
        g = _gen(seed, 4)
        step = max(1, (1 << 25) // k)
        for a in range(0, n, step):
            w = _randn((min(step, n - a), k), g).mul_(0.02)
            c, e = _mx(w)
            c = (c | (torch.signbit(w).to(torch.uint8) << 3).view(c.shape)).view(w.shape)
            s["w"][a:a + step] = c[:, 0::2] | (c[:, 1::2] << 4)
            bytes_[a:a + step] = (e + 127).to(torch.uint8)
        s["wsc"] = _tile(bytes_)
        s["x"] = _hidden(m, k, _gen(seed, 1)).to(t)
        s["y"] = torch.empty((m, n), dtype=TYPES[case["out"]], device="cuda")
        s["ws"] = torch.empty(-(-m * k // 2 // 256) * 256 + _scale_bytes(m, k), dtype=torch.uint8, device="cuda")
    else:
        v, g = case["v"], _gen(seed, 5)
        x = _randn((m, v), g).mul_(2.5)
        hot = torch.randint(0, v, (m, 8), generator=g, device="cuda")
        more = 6 + 2 * _randn((m, 8), g)
        for j in range(8):                                      # a few likely tokens
            x.scatter_add_(1, hot[:, j:j + 1], more[:, j:j + 1])
        tokens = torch.where(torch.rand((m,), generator=g, device="cuda") < 0.7, hot[:, 0],
                             torch.randint(0, v, (m,), generator=g, device="cuda"))
        if case["masked"]:
            x.masked_fill_(torch.rand((m, v), generator=g, device="cuda") < 0.5, -math.inf)
            x[5::16] = -math.inf                                # rows whose mask leaves nothing
            tokens[3::16] = -1                                  # rows of padding: no token asked for
        s["logits"] = x.to(t)
        s["tokens"] = tokens.to(torch.int32)
        s["out"] = (torch.empty(m, device="cuda"), torch.empty(m, device="cuda"),
                    torch.empty((m, case["top"]), dtype=torch.int32, device="cuda"),
                    torch.empty((m, case["top"]), device="cuda"))
    return s


# ---------------------------------------------------------------------------------------
# The operators
# ---------------------------------------------------------------------------------------
def run(s):
    return {"norm": _norm, "quantize": _quantize, "product": _product, "logprobs": _logprobs}[s["op"]](s)


def _norm(s):
    m, k, r = s["m"], s["k"], s["r"]
    out = {}
    if own:
        import q8_block_quantized_act_gb300 as q8
        if s["layout"] == "q8_1":
            q8.rmsnorm_q8_1(s["x"], s["w"], EPS, residual=r, residual_out=s["r_out"], out=(s["q"], s["d"]))
            torch.mul(s["q"].view(s["values"].shape), s["d"].unsqueeze(-1), out=s["values"])
            out["values"] = s["values"]
        else:
            q8.rmsnorm_q8_1_mmq(s["x"], s["w"], EPS, residual=r, residual_out=s["r_out"], out=(s["q"], s["d"]))
            out["quants"], out["scales"] = s["q"].view(torch.float16), s["d"][:, :m]
        if r is not None:
            out["residual"] = s["r_out"]
        return out
    h = s["x"].float()
    if r is not None:
        h = h + r.float()
        out["residual"] = h.to(s["x"].dtype)
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["w"].float()
    b = y.view(m, k // QK, QK)
    d = b.abs().amax(-1, keepdim=True) / 127
    t = torch.where(d > 0, b / d, torch.zeros_like(b))
    q = ((t.abs() + 0.5).floor().copysign(t)).clamp(-127, 127)
    if s["layout"] == "q8_1":
        out["values"] = (q * d).half()
    else:
        out["quants"], out["scales"] = q.half().view(m, k), d.view(m, -1).t()
    return out


def _quantize(s):
    if own:
        import q8_block_quantized_act_gb300 as q8
        q8.quantize_mxfp4(s["x"], out=(s["codes"], s["scales"]))
        return q8.dequant_mxfp4(s["codes"], s["scales"], out=s["values"])
    return _mx_values(s["x"].float()).bfloat16()


def _product(s):
    if own:
        import q8_block_quantized_act_gb300 as q8
        return q8.gemm_mxfp4(s["w"], s["wsc"], s["x"], ws=s["ws"], out=s["y"])
    n, k = s["n"], s["k"]
    c = torch.stack((s["w"] & 15, s["w"] >> 4), -1).view(n, k // QK, QK).int()
    mag = _magnitudes(c.device)
    w = torch.cat((mag, -mag))[c] * _pow2(_untile(s["wsc"], n, k // QK).int() - 127).unsqueeze(-1)
    return (_mx_values(s["x"].float()) @ w.view(n, k).t()).to(s["y"].dtype)


def _logprobs(s):
    x, tokens, top = s["logits"], s["tokens"], s["top"]
    if own:
        import q8_block_quantized_act_gb300 as q8
        lp, h, ids, tlp = q8.logprobs(x, tokens, top=top, out=s["out"])
        return {"logprob": lp, "entropy": h, "ids": ids, "top": tlp}
    x = x.float()
    mx = x.amax(-1, keepdim=True)
    empty = mx == -math.inf
    z = torch.where(empty, x, x - mx)                  # <= 0, -inf where masked
    e = torch.exp(z)
    total = e.sum(-1, keepdim=True)
    lse = torch.where(empty, torch.zeros_like(mx), total.log())
    h = torch.where(empty, torch.zeros_like(mx), lse - torch.where(e > 0, z * e, e).sum(-1, keepdim=True) / total)
    at = z.gather(1, tokens.clamp(min=0).long().unsqueeze(-1)) - lse
    lp = torch.where(tokens < 0, torch.zeros_like(mx[:, 0]), at[:, 0])
    best, ids = torch.sort(x, dim=-1, descending=True, stable=True)     # equal logits: the lowest index first
    best, ids = best[:, :top], ids[:, :top]
    ids = torch.where(best == -math.inf, torch.full_like(ids, -1), ids)
    return {"logprob": lp, "entropy": h[:, 0], "ids": ids.int(), "top": torch.where(empty, best, best - mx) - lse}


# ---------------------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------------------
def work(case):
    op, m = case["op"], case["m"]
    size = SIZE[case["type"]]
    if op == "norm":
        k = case["k"]
        q = 1 if case["layout"] == "q8_1" else 2
        return {"bytes": m * k * (size * (3 if case["residual"] else 1) + q + 4 / QK) + k * size, "flops": 8 * m * k}
    if op == "quantize":
        return {"bytes": m * case["k"] * (size + 17 / 32 + 2), "flops": 4 * m * case["k"]}
    if op == "product":
        n, k = case["n"], case["k"]
        return {"bytes": n * k * 17 / 32 + m * k * size + m * n * SIZE[case["out"]], "flops": 2 * m * n * k}
    v, top = case["v"], case["top"]
    return {"bytes": m * v * size + m * (12 + 8 * top), "flops": 6 * m * v}


# ---------------------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------------------
def _e2m1_64(x):
    """Blocks of 32 of a float64 array [rows][k] to the nearest values of the MXFP4 grid."""
    grid = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
    grid = torch.from_numpy(grid).to(x.device)
    b = x.reshape(-1, QK)
    top = b.abs().amax(1, keepdim=True)
    unit = torch.where(top > 0, torch.exp2(torch.floor(torch.log2(torch.where(top > 0, top, torch.ones_like(top)))) - 2),
                       torch.ones_like(top))
    unit = torch.where(top / unit >= 8, unit * 2, torch.where((top > 0) & (top / unit < 4), unit / 2, unit))
    a = b.abs() / unit
    up = torch.searchsorted(grid, a.contiguous()).clamp(1, 7)      # grid[up - 1] < a <= grid[up]
    lo, hi = grid[up - 1], grid[up]
    nearer = (a - lo > hi - a) | ((a - lo == hi - a) & (up % 2 == 0))
    return (torch.where(nearer, hi, lo) * unit * torch.sign(b)).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    op, m = case["op"], case["m"]
    if op == "norm":
        out = {}
        h = s["x"].double()
        if s["r"] is not None:
            h = h + s["r"].double()
            out["residual"] = h
        y = s["w"].double() * h / torch.sqrt(h.square().sum(1, keepdim=True) / case["k"] + EPS)
        b = y.reshape(m, -1, QK)
        d = b.abs().max(2, keepdim=True).values / 127
        q = torch.trunc(b / d + torch.sign(b) / 2)
        if case["layout"] == "q8_1":
            out["values"] = q * d
        else:
            out["quants"], out["scales"] = q.reshape(m, -1), d[..., 0].T
        return out
    if op == "quantize":
        rows = max(1, (1 << 25) // case["k"])
        return torch.cat([_e2m1_64(a.double()) for a in s["x"].split(rows)])
    if op == "product":
        n, k = case["n"], case["k"]
        x = _e2m1_64(s["x"].double()).T
        at = torch.arange(n, device="cuda")
        blocks = torch.arange(k // QK, device="cuda")
        # where the byte of row r and block b stands
        place = ((at // 128 * (k // 128)).unsqueeze(1) + blocks // 4) * 512 + (
            at % 32 * 16 + at % 128 // 32 * 4).unsqueeze(1) + blocks % 4
        table = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12, 0, -1, -2, -3, -4, -6, -8, -12], dtype=torch.float64, device="cuda") / 2
        parts = []
        step = max(1, (1 << 25) // k)
        for a in range(0, n, step):
            w = s["w"][a:a + step].long()
            v = torch.empty((w.shape[0], k), dtype=torch.float64, device="cuda")
            v[:, 0::2], v[:, 1::2] = table[w % 16], table[w // 16]
            sc = torch.pow(2.0, s["wsc"][place[a:a + step]].double() - 127)
            parts.append((v * sc.repeat_interleave(QK, 1)) @ x)
        return torch.cat(parts).T
    out = {"logprob": [], "entropy": [], "top": []}
    for row, token in zip(s["logits"].double().split(1), s["tokens"].tolist()):
        row = row[0]
        live = row[row > -math.inf]
        best = torch.full((case["top"],), -math.inf, dtype=torch.float64, device="cuda")
        if live.numel():
            lp = live - torch.logsumexp(live, 0)
            got = torch.sort(lp, descending=True).values[:case["top"]]
            best[:got.numel()] = got
            out["entropy"].append(-(lp * lp.exp()).sum())
            asked = row[token] - torch.logsumexp(live, 0)
        else:
            out["entropy"].append(torch.zeros((), dtype=torch.float64, device="cuda"))
            asked = row[0]
        out["logprob"].append(asked if token >= 0 else torch.zeros_like(asked))
        out["top"].append(best)
    return {"ids": None, **{n: torch.stack(v) for n, v in out.items()}}
