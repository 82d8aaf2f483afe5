"""Plain 64-bit forms of the paged cache's append and attention, with the error that their f32
arithmetic and roundings may have.  torch on the CPU; nothing of the library's code."""
import math
import random

import torch

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def half(t):
    """The largest relative error of one rounding to t."""
    return torch.finfo(t).eps / 2


def tiny(t):
    """The largest absolute error of one rounding to t below its normal range."""
    return torch.finfo(t).tiny * torch.finfo(t).eps / 2


class Batch:
    """Sequences given as (positions before, new tokens), their pages shuffled over a cache with some to
    spare.  Everything that no position uses holds `filler`."""

    def __init__(self, seqs, hk, d, page, t, seed=0, filler=math.nan, spare=2, width=None, first=0, pad=0):
        rng = random.Random(seed)
        g = torch.Generator().manual_seed(seed)
        self.seqs, self.hk, self.d, self.page, self.t = seqs, hk, d, page, t
        used = [-(-(c + n) // page) for c, n in seqs]
        self.pages = sum(used) + spare
        ids = list(range(self.pages))
        rng.shuffle(ids)
        self.width = width or max(max(used), 1)
        self.table = torch.full((len(seqs), self.width), -1, dtype=torch.int32)
        for b, n in enumerate(used):
            for j in range(n):
                self.table[b, j] = ids.pop()
        self.lens = torch.tensor([c + n for c, n in seqs], dtype=torch.int32)
        starts = [first]
        for _, n in seqs:
            starts.append(starts[-1] + n)
        self.starts = torch.tensor(starts, dtype=torch.int32)
        self.m = starts[-1] + pad
        self.k = torch.full((self.pages, hk, page, d), filler, dtype=t)
        self.v = torch.full((self.pages, hk, page, d), filler, dtype=t)
        for b, (c, n) in enumerate(seqs):
            for p in range(c + n):
                at, slot = int(self.table[b, p // page]), p % page
                if at < 0:
                    continue
                self.k[at, :, slot] = torch.randn((hk, d), generator=g).to(t)
                self.v[at, :, slot] = torch.randn((hk, d), generator=g).to(t)
        self.g = g

    def randn(self, *shape, t=None):
        return torch.randn(shape, generator=self.g).to(t or self.t)

    def cuda(self):
        return [x.cuda() for x in (self.k, self.v, self.table, self.starts, self.lens)]

    def tokens(self):
        """(row, sequence, position) of every new token."""
        for b in range(len(self.seqs)):
            s0, s1 = int(self.starts[b]), int(self.starts[b + 1])
            for r in range(s0, s1):
                yield r, b, int(self.lens[b]) - s1 + r

    def place(self, b, p):
        """(page, slot) of a position, or None."""
        if p < 0 or p // self.page >= self.width:
            return None
        at = int(self.table[b, p // self.page])
        return (at, p % self.page) if 0 <= at < self.pages else None


def rotated(x, pos, inv_freq, interleaved):
    """x f64 [tokens, heads, d], pos f64 [tokens] -> (values, sum of the magnitudes that each is made of)."""
    n = len(inv_freq)
    out, size = x.clone(), x.abs()
    if n == 0:
        return out, size
    ang = pos[:, None] * torch.as_tensor(inv_freq, dtype=torch.float64)
    c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
    i = torch.arange(n)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    a, b = x[..., ia], x[..., ib]
    out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
    size[..., ia] = size[..., ib] = a.abs() + b.abs()
    return out, size


# Of a rotated value, relative to |a| + |b|: the angle rounded to f32 (2^-24 of half a turn: 2^-22.3), sine
# and cosine (2 units of 2^-24 each, and the part of a turn that 32 bits leave out), two products and a sum.
ROTATION = 2.0 ** -22.3 + 2 * 2.0 ** -24 + 2.0 ** -29 + 3 * 2.0 ** -24


def append(batch, q, k, v, inv_freq, interleaved, t):
    """What the cache and the queries hold afterwards: (q64, q_tol), (k64, k_tol), v; rows of q that belong to
    no sequence and places that nothing is written to are NaN in the 64-bit arrays."""
    pos = torch.zeros(q.shape[0], dtype=torch.float64)
    kc = torch.full(batch.k.shape, math.nan, dtype=torch.float64)
    ktol = torch.zeros(batch.k.shape, dtype=torch.float64)
    vc = batch.v.clone()
    mine = torch.zeros(q.shape[0], dtype=torch.bool)
    todo = list(batch.tokens())
    for r, b, p in todo:
        pos[r], mine[r] = p, True
    q64, qs = rotated(q.double(), pos, inv_freq, interleaved)
    k64, ks = rotated(k.double(), pos, inv_freq, interleaved)
    tol = lambda x, s: ROTATION * s * (1 + half(t)) + half(t) * x.abs() + tiny(t)          # noqa: E731
    q64[~mine] = math.nan
    for r, b, p in todo:
        at = batch.place(b, p)
        if at is not None and p < int(batch.lens[b]):
            kc[at[0], :, at[1]], ktol[at[0], :, at[1]] = k64[r], tol(k64[r], ks[r])
            vc[at[0], :, at[1]] = v[r].to(t)
    return (q64, tol(q64, qs)), (kc, ktol), vc


def attention(batch, q, scale, window, out_t):
    """(out64, tolerance) [m, hq, d]; rows that belong to no sequence are NaN."""
    m, hq, d = q.shape
    group = hq // batch.hk
    c = batch.t
    out = torch.full((m, hq, d), math.nan, dtype=torch.float64)
    tol = torch.zeros((m, hq, d), dtype=torch.float64)
    U = 2.0 ** -23            # of f32 sums on the tensor cores, which may cut where others round
    for b in range(len(batch.seqs)):
        rows = [(r, p) for r, bb, p in batch.tokens() if bb == b]
        if not rows:
            continue
        keys = [(p, batch.place(b, p)) for p in range(int(batch.lens[b]))]
        keys = [(p, at) for p, at in keys if at is not None]
        r = torch.tensor([x for x, _ in rows])
        pos = torch.tensor([x for _, x in rows], dtype=torch.int64)[:, None]
        kp = torch.tensor([p for p, _ in keys], dtype=torch.int64)[None]
        at = torch.tensor([a for _, (a, _) in keys], dtype=torch.int64)
        slot = torch.tensor([s for _, (_, s) in keys], dtype=torch.int64)
        seen = kp <= pos
        if window:
            seen &= kp > pos - window
        for h in range(batch.hk):
            k, v = batch.k[at, h, slot].double(), batch.v[at, h, slot].double()      # [keys, d]
            for j in range(h * group, (h + 1) * group):
                x = q[r, j].double()
                s = torch.where(seen, scale * x @ k.T, torch.full(seen.shape, -math.inf, dtype=torch.float64))
                mx = s.max(1, keepdim=True).values if keys else torch.full((len(rows), 1), -math.inf)
                p = torch.where(seen, torch.exp(s - torch.where(mx == -math.inf, torch.zeros_like(mx), mx)),
                                torch.zeros_like(s))
                total = p.sum(1, keepdim=True)
                w = torch.where(total > 0, p / torch.where(total > 0, total, torch.ones_like(total)), p)
                # values that a row does not see do not count, whatever they are
                clean = torch.where(seen.any(0)[:, None], v, torch.zeros_like(v)) if keys else v
                if not torch.isfinite(clean).all():
                    o = torch.stack([(w[i, seen[i]][:, None] * v[seen[i]]).sum(0) for i in range(len(rows))])
                    a = torch.stack([(w[i, seen[i]][:, None] * v[seen[i]].abs()).sum(0) for i in range(len(rows))])
                    top = torch.stack([v[seen[i]].abs().amax(0) if bool(seen[i].any()) else torch.zeros(d) for i in range(len(rows))])
                else:
                    o, a = w @ clean, w @ clean.abs()
                    top = clean.abs().amax(0, keepdim=True) if keys else torch.zeros((1, d))
                n = seen.sum(1, keepdim=True).double()
                size = torch.where(seen, scale * x.abs() @ k.abs().T, torch.zeros(seen.shape, dtype=torch.float64))
                size = torch.nan_to_num(size, 0.0, 0.0, 0.0).amax(1, keepdim=True) if keys else torch.zeros((len(rows), 1))
                ds = (d + 4) * U * size                      # of a score, and so relative of a weight
                rel = half(c) + 2 * ds + (2 * n + 16) * U    # a weight's rounding; sums above and below
                out[r, j] = o
                tol[r, j] = (a * rel + n * tiny(c) * top) * (1 + half(out_t)) + half(out_t) * o.abs() + tiny(out_t)
    return out, tol


def close(got, want, tol, what=""):
    """got within tol of want; NaN and infinities where want has them."""
    got = got.detach().cpu().double()
    fin = torch.isfinite(want)
    assert torch.equal(torch.isnan(got) & ~fin, torch.isnan(want)), f"{what}: NaN elsewhere"
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities"
    err = torch.where(fin, (got - want).abs(), torch.zeros_like(want))
    bad = fin & ~(err <= tol)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off; first {i}: {got[i]} for {want[i]}, tolerance {tol[i]}")
