"""The paged key/value cache of a decoder and the attention over it, and how they are measured.

Two operators, as a serving step meets them between its projections:

  append     rotation of the new tokens' queries and keys by their positions; keys and values
             into the pages of the cache, queries into the attention's type
  attention  causal attention of the new tokens (one a sequence, a few, or a chunk of a prompt)
             over the cache, grouped query heads, optionally over a window of positions

`own` selects the framework's kernels; otherwise each operator is computed from elementary
torch operations in 32 bits.
"""
import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
BASE = 500000.0                     # of the rotation's frequencies

# A batch is `seqs` sequences.  Each has up to `ctx` tokens in the cache already and brings up to
# `new` more; the first has exactly as many, the others as many (spread "even") or anything from a
# few on (spread "ragged").


# ---------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------
def _append(name, seqs, new, ctx, spread, hq, hk, d, page, src, kind, pairs="halves", shape=0):
    return dict(name=name, op="append", seqs=seqs, new=new, ctx=ctx, spread=spread, hq=hq, hk=hk, d=d, page=page,
                src=src, type=kind, pairs=pairs, shape=shape)


def _attention(name, seqs, new, ctx, spread, hq, hk, d, page, kind, window=0, shape=0):
    return dict(name=name, op="attention", seqs=seqs, new=new, ctx=ctx, spread=spread, hq=hq, hk=hk, d=d, page=page,
                type=kind, window=window, shape=shape)


def listed():
    return [
        # one decoded token behind the fused projection: latency
        _append("append 1 token f32 to f16", 1, 1, 4096, "even", 32, 8, 128, 64, "f32", "f16"),
        # speculative tokens of a ragged batch, neighbouring values rotated as pairs, narrow heads
        _append("append 21 sequences x 7 bf16", 21, 7, 1000, "ragged", 20, 4, 64, 16, "bf16", "bf16", "neighbours"),
        # the largest prompt
        _append("append 8191 tokens bf16", 1, 8191, 0, "even", 32, 8, 128, 128, "bf16", "bf16"),
        # one decoded token of one user: latency
        _attention("decode 1 x 4096 f16", 1, 1, 4096, "even", 32, 8, 128, 64, "f16"),
        # one user's token over a long document: one sequence has to fill the GPU
        _attention("decode 1 x 131071 bf16", 1, 1, 131071, "even", 32, 8, 128, 64, "bf16"),
        # a serving batch at ordinary lengths
        _attention("decode 64 x 8192 ragged bf16", 64, 1, 8192, "ragged", 32, 8, 128, 16, "bf16"),
        # many short conversations of a small model without grouped heads
        _attention("decode 190 x 600 ragged f16", 190, 1, 600, "ragged", 12, 12, 64, 16, "f16"),
        # speculative tokens being verified
        _attention("verify 16 x 5 at 6000 f16", 16, 5, 6000, "ragged", 28, 4, 128, 32, "f16"),
        # the next chunk of a long prompt
        _attention("chunk 509 at 16384 f16", 1, 509, 16384, "even", 32, 8, 128, 64, "f16"),
        # prompts and single tokens in one batch
        _attention("mixed 25 x 2000 bf16", 25, 2000, 3000, "ragged", 32, 4, 128, 32, "bf16"),
        # local attention layers of a long prompt
        _attention("window 1024 of 8000 f16", 1, 8000, 0, "even", 64, 8, 64, 64, "f16", window=1024),
        # the largest prompt
        _attention("prefill 8192 bf16", 1, 8192, 0, "even", 32, 8, 128, 128, "bf16"),
    ]


HEADS = ((32, 8, 128), (32, 4, 128), (28, 4, 128), (8, 1, 128), (6, 2, 128), (64, 8, 64), (12, 12, 64), (20, 4, 64))


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = work(listed()[-1])["flops"]
    while True:
        hq, hk, d = rng.choice(HEADS)
        page, kind = rng.choice((16, 32, 64, 128)), rng.choice(("f16", "bf16"))
        shape = rng.randrange(1 << 20)
        if rng.random() < 0.3:
            c = _append("", _log(rng, 1, 128), _log(rng, 1, 8191), _log(rng, 1, 8192) - 1, rng.choice(("even", "ragged")),
                        hq, hk, d, page, rng.choice(tuple(TYPES)), kind, rng.choice(("halves", "neighbours")), shape)
            if c["seqs"] * c["new"] > 8191 or c["seqs"] * (c["new"] + c["ctx"]) > 1 << 17:
                continue
        else:
            new = 1 if rng.random() < 0.4 else _log(rng, 2, 8192)
            c = _attention("", _log(rng, 1, 256), new, _log(rng, 1, 131072) - 1, rng.choice(("even", "ragged")), hq, hk, d,
                           page, kind, _log(rng, 16, 8192) if rng.random() < 0.25 else 0, shape)
            if c["seqs"] * new > 16384 or c["seqs"] * (new + c["ctx"]) > 1 << 18 or work(c)["flops"] > most:
                continue
        del c["name"]
        return c


def lengths(case):
    """Per sequence: (tokens in the cache before the call, new tokens)."""
    rng = random.Random(case["shape"] * 1009 + case["seqs"])
    out = [(case["ctx"], case["new"])]
    for _ in range(case["seqs"] - 1):
        if case["spread"] == "even":
            out.append((case["ctx"], case["new"]))
        else:
            out.append((_log(rng, max(1, case["ctx"] // 16), max(1, case["ctx"])), _log(rng, 1, case["new"])))
    return out


# ---------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------
def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 16 + salt)
    return g


def _randn(shape, g, t):
    """Unit normal values of type t, made in parts."""
    out = torch.empty(shape, dtype=t, device="cuda")
    for part in out.view(-1).split(1 << 27):
        part.copy_(torch.randn(part.shape, generator=g, device="cuda"))
    return out


def _inputs(case, seed):
    s = dict(case)
    hq, hk, d, page, t = case["hq"], case["hk"], case["d"], case["page"], TYPES[case["type"]]
    lens = lengths(case)
    total = [c + n for c, n in lens]
    used = [-(-n // page) for n in total]
    pages = sum(used) + 3                                    # some stay free
    g = torch.Generator()
    g.manual_seed(seed * 16 + 1)
    order = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(used)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    starts = [0]
    for _, n in lens:
        starts.append(starts[-1] + n)
    m = starts[-1]
    s["m"], s["total"], s["starts_list"] = m, total, starts
    s["table"] = table.cuda()
    s["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    s["lens"] = torch.tensor(total, dtype=torch.int32, device="cuda")
    s["kc"] = _randn((pages, hk, page, d), _gen(seed, 2), t)
    s["vc"] = _randn((pages, hk, page, d), _gen(seed, 3), t)
    if case["op"] == "append":
        qkv = _randn((m, hq + 2 * hk, d), _gen(seed, 4), TYPES[case["src"]])     # the fused projection's rows
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        s["inv_freq"] = BASE ** (-torch.arange(0, d, 2, dtype=torch.float64) / d).cuda()
        s["out"] = torch.empty((m, hq, d), dtype=t, device="cuda")
    else:
        # queries of one head in eight look for something: their scores spread twice as wide
        q = _randn((m, hq, d), _gen(seed, 4), t)
        q[:, ::8] *= 2
        s["q"] = q
        s["out"] = torch.empty_like(q)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import q8_block_quantized_act_gb300 as q8
        s["kv"] = q8.PagedKV(s["kc"], s["vc"], s["table"], s["starts"], s["lens"])
        if case["op"] == "append":
            s["turns"] = q8.rope_turns(s["inv_freq"])
        else:
            s["ws"] = q8.attention_workspace(s["kv"], case["hq"])
    return s


# ---------------------------------------------------------------------------------------
# The operators
# ---------------------------------------------------------------------------------------
def run(s):
    return _run_append(s) if s["op"] == "append" else _run_attention(s)


def _run_append(s):
    if own:
        import q8_block_quantized_act_gb300 as q8
        q = q8.append_kv(s["kv"], s["q"], s["k"], s["v"], turns=s["turns"], interleaved=s["pairs"] == "neighbours",
                         out=s["out"])
        return {"q": q, "k": s["kc"], "v": s["vc"]}
    t, page = s["kc"].dtype, s["page"]
    starts, lens = s["starts"].long(), s["lens"].long()
    token = torch.arange(s["m"], device="cuda")
    seq = (token.unsqueeze(1) >= starts[1:]).sum(1)
    pos = lens[seq] - starts[seq + 1] + token
    angle = pos.double().unsqueeze(1) * s["inv_freq"]
    cos, sin = angle.cos().float().unsqueeze(1), angle.sin().float().unsqueeze(1)

    def rotate(x):
        x = x.float()
        if s["pairs"] == "halves":
            a, b = x.chunk(2, -1)
            return torch.cat((a * cos - b * sin, b * cos + a * sin), -1).to(t)
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2).to(t)

    where, slot = s["table"][seq, pos // page].long(), pos % page
    s["kc"][where, :, slot] = rotate(s["k"])
    s["vc"][where, :, slot] = s["v"].float().to(t)
    return {"q": rotate(s["q"]), "k": s["kc"], "v": s["vc"]}


def _run_attention(s):
    if own:
        import q8_block_quantized_act_gb300 as q8
        return q8.attention(s["kv"], s["q"], window=s["window"], max_new=s["new"], ws=s["ws"], out=s["out"])
    hq, hk, d, page, window = s["hq"], s["hk"], s["d"], s["page"], s["window"]
    group = hq // hk
    out = torch.empty_like(s["q"])
    for b, n in enumerate(s["total"]):
        lo, hi = s["starts_list"][b:b + 2]
        at = s["table"][b, :-(-n // page)].long()
        k = s["kc"][at].transpose(0, 1).reshape(hk, -1, d)[:, :n].float()
        v = s["vc"][at].transpose(0, 1).reshape(hk, -1, d)[:, :n].float()
        step = max(1, (1 << 29) // (hq * n))
        for a in range(lo, hi, step):
            e = min(a + step, hi)
            q = s["q"][a:e].float().view(e - a, hk, group, d).transpose(0, 1).reshape(hk, -1, d)
            score = (q @ k.transpose(1, 2)).view(hk, e - a, group, n) * d ** -0.5
            pos = torch.arange(a, e, device="cuda").view(1, -1, 1, 1) + (n - hi)
            key = torch.arange(n, device="cuda")
            hidden = key > pos
            if window:
                hidden = hidden | (key <= pos - window)
            score.masked_fill_(hidden, -math.inf)
            p = torch.exp(score - score.amax(-1, keepdim=True))
            o = (p.view(hk, -1, n) @ v).view(hk, e - a, group, d) / p.sum(-1, keepdim=True)
            out[a:e] = o.transpose(0, 1).reshape(e - a, hq, d)
    return out


# ---------------------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------------------
def work(case):
    hq, hk, d, size = case["hq"], case["hk"], case["d"], SIZE[case["type"]]
    lens = lengths(case)
    m = sum(n for _, n in lens)
    if case["op"] == "append":
        values = m * (hq + 2 * hk) * d
        return {"bytes": values * (SIZE[case["src"]] + size) + 4 * d, "flops": 6 * m * (hq + hk) * d // 2}
    pairs = keys = 0
    for ctx, n in lens:
        w = case["window"] or ctx + n
        full = max(0, min(n, w - ctx))                       # tokens whose window still reaches back to the start
        pairs += full * ctx + full * (full + 1) // 2 + (n - full) * w
        keys += ctx + n - max(0, ctx + 1 - w)
    return {"bytes": (2 * keys * hk + 2 * m * hq) * d * size, "flops": 4 * pairs * hq * d}


# ---------------------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------------------
def exact(case, seed):
    s = _inputs(case, seed)
    hq, hk, d, page = case["hq"], case["hk"], case["d"], case["page"]
    if case["op"] == "append":
        out = {"q": torch.empty((s["m"], hq, d), dtype=torch.float64, device="cuda"),
               "k": s["kc"].double(), "v": s["vc"].double()}
        first = 0
        for (ctx, n), row in zip(lengths(case), s["table"].tolist()):
            pos = torch.arange(ctx, ctx + n, device="cuda")
            turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                               pos.double()[:, None] * s["inv_freq"][None])[:, None]

            def rotated(x):
                x = x[first:first + n].double()
                pair = (x[..., :d // 2], x[..., d // 2:]) if case["pairs"] == "halves" else (x[..., ::2], x[..., 1::2])
                z = torch.complex(*pair) * turn
                return torch.cat((z.real, z.imag), -1) if case["pairs"] == "halves" else torch.view_as_real(z).flatten(-2)

            out["q"][first:first + n] = rotated(s["q"])
            k, v = rotated(s["k"]), s["v"][first:first + n].double()
            for p in range(ctx // page, (ctx + n - 1) // page + 1):              # page by page
                a, e = max(ctx, p * page), min(ctx + n, (p + 1) * page)
                out["k"][row[p], :, a - p * page:e - p * page] = k[a - ctx:e - ctx].transpose(0, 1)
                out["v"][row[p], :, a - p * page:e - p * page] = v[a - ctx:e - ctx].transpose(0, 1)
            first += n
        return out
    if work(case)["flops"] > 3e12:
        return None
    out = torch.empty((s["m"], hq, d), dtype=torch.float64, device="cuda")
    first = 0
    for (ctx, n), row in zip(lengths(case), s["table"]):
        pages = row[:(ctx + n + page - 1) // page].long()
        for h in range(hk):
            k = s["kc"][pages, h].reshape(-1, d)[:ctx + n].double()
            v = s["vc"][pages, h].reshape(-1, d)[:ctx + n].double()
            for j in range(h * hq // hk, (h + 1) * hq // hk):
                for a in range(0, n, 4096):
                    e = min(n, a + 4096)
                    # the keys that the rows a..e see at all
                    lo = max(0, ctx + a + 1 - case["window"]) if case["window"] else 0
                    hi = ctx + e
                    z = s["q"][first + a:first + e, j].double() @ k[lo:hi].T / math.sqrt(d)
                    back = (torch.arange(ctx + a, ctx + e, device="cuda")[:, None] -
                            torch.arange(lo, hi, device="cuda")[None])
                    seen = back >= 0
                    if case["window"]:
                        seen &= back < case["window"]
                    z = torch.where(seen, z, torch.full_like(z, -math.inf))
                    out[first + a:first + e, j] = torch.exp(z - torch.logsumexp(z, 1, keepdim=True)) @ v[lo:hi]
        first += n
    return out
