"""attention where a CTA takes many key tiles of both row tiles, several units one after another, or a part of a
sequence that many share; sums that show each part."""
import pytest
import torch

import paged_ref as ref
import q8_block_quantized_act_gb300 as q8
from gpu_util import device_ok, ensure_built


def check(batch, hq, window=0, max_new=None, out_t=None):
    q = batch.randn(batch.m, hq, batch.d)
    out_t = out_t or batch.t
    want, tol = ref.attention(batch, q, batch.d ** -0.5, window, out_t)
    got = q8.attention(q8.PagedKV(*batch.cuda()), q.cuda(), window=window, max_new=max_new, dtype=out_t)
    device_ok()
    ref.close(got, want, tol)


# 128 values a head.  More than 152 units of 256 rows that see five key tiles and more, so that most have tiles with nothing
# masked in them for both of their row tiles, and a CTA has two units and more.
FULL = [
    ([(1000, 380)], 128, 64),                                                    # a sequence of 192 units
    ([(500, 340)], 144, 48),                                                     # queries row by row: 3 heads of a group
    ([(700, 130), (0, 640), (900, 1), (300, 257), (0, 0)], 96, 48),              # by length, also short ones
    ([(640, 140)] * 6 + [(i, 1) for i in range(30)], 64, 16),                    # more than 32 sequences
]


@pytest.mark.gpu
@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("seqs,hq,hk", FULL, ids=["one", "group of 3", "by length", "many sequences"])
def test_full_units(seqs, hq, hk, t):
    ensure_built()
    check(ref.Batch(seqs, hk, 128, 64, ref.TYPES[t], seed=hq), hq)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_full_units_behind_a_window(d):
    ensure_built()
    check(ref.Batch([(700, 300), (1200, 200)], 48, d, 16, torch.float16, seed=d), 96, window=650)


# ---------------------------------------------------------------------------------------
# Equal scores, and values that say which 16 positions they are of: weights, products and sums are whole numbers (times a power
# of two), so an output is a quotient of two of them, and 16 positions that are missing or counted twice are seen.
# ---------------------------------------------------------------------------------------
def counting(seqs, d, page, t):
    """seqs: (positions, new tokens) -> caches and table of one head, what column of values each position has."""
    most = max(n for n, _ in seqs)
    pages = [-(-n // page) for n, _ in seqs]
    order = torch.randperm(sum(pages), generator=torch.Generator().manual_seed(most)).split(pages)
    table = torch.full((len(seqs), max(pages)), -1, dtype=torch.int32)
    v = torch.zeros((sum(pages), 1, page, d), dtype=t)
    for b, ((n, _), at) in enumerate(zip(seqs, order)):
        table[b, :pages[b]] = at.to(torch.int32)
        x = torch.zeros((pages[b] * page, d), dtype=t)
        x[torch.arange(n), columns(n, b, d)] = 1
        v[at] = x.view(pages[b], 1, page, d)
    k = torch.zeros_like(v)
    return k, v, table


def columns(n, b, d):
    return (torch.arange(n) // 16 + b) % d


def expected(seqs, d, without=None):
    """[new tokens, d]: the share of the positions 0 .. p whose values are in each column; without (from, to) of them."""
    rows = []
    for b, (n, new) in enumerate(seqs):
        if not new:
            continue
        there = torch.ones(n, dtype=torch.float64)
        if without:
            there[without[0]:without[1]] = 0
        counts = torch.zeros((n, d), dtype=torch.float64)
        counts[torch.arange(n), columns(n, b, d)] = there
        before = counts[:n - new].sum(0)
        seen = (before + counts[n - new:].cumsum(0))
        rows.append(seen / torch.arange(n - new + 1, n + 1)[:, None])
    return torch.cat(rows)


# Whole numbers below 2^24: what is rounded is the quotient, once as 1 / sum and once as a product.
def tolerance(want):
    return 2.0 ** -22 * want


LONG = [
    [(20000, 5)], [(131071, 5)], [(131072, 1)], [(70000, 40)],
    [(9000, 5), (40, 5), (33000, 3), (1, 1), (5000, 0)],
    [(20000, 5)] + [(30 + i, i % 4) for i in range(40)],
    [(100 + i, 1) if i % 13 else (30000 + i, 5) for i in range(50)],
]


@pytest.mark.gpu
@pytest.mark.parametrize("d,page", [(64, 16), (128, 64)])
@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("group", [1, 4, 20])
@pytest.mark.parametrize("seqs", LONG, ids=["20000", "131071", "decode 131072", "70000", "few", "many", "many long"])
def test_every_part_counts_once(seqs, group, t, d, page):
    """Of up to 16 rows in the kernel for few rows, of as many as there are in the one for chunks."""
    ensure_built()
    t = ref.TYPES[t]
    k, v, table = counting(seqs, d, page, t)
    i32 = dict(dtype=torch.int32, device="cuda")
    starts = torch.tensor([0] + [n for _, n in seqs], **i32).cumsum(0).to(torch.int32)
    kv = q8.PagedKV(k.cuda(), v.cuda(), table.cuda(), starts, torch.tensor([n for n, _ in seqs], **i32))
    m = int(starts[-1])
    q = torch.randn((m, group, d), device="cuda").to(t)
    want = expected(seqs, d)[:, None].expand(-1, group, -1)
    for max_new in (1, None):
        got = q8.attention(kv, q, max_new=max_new, dtype=torch.float32)
        device_ok()
        ref.close(got, want, tolerance(want), f"max_new {max_new}")


@pytest.mark.parametrize("seqs", LONG, ids=str)
def test_a_missing_part_would_be_seen(seqs):
    """The form above with 16 positions left out is beyond the tolerance of what it is with all of them."""
    for d in (64, 128):
        want = expected(seqs, d)
        for at in (0, 16):
            without = expected(seqs, d, (at, at + 16))
            assert bool(((without - want).abs() > tolerance(want)).any(1).all()) or at >= min(n for n, new in seqs if new)
        ref.close(want, want, tolerance(want))
        with pytest.raises(AssertionError):
            ref.close(expected(seqs, d, (0, 16)), want, tolerance(want))


@pytest.mark.gpu
@pytest.mark.parametrize("max_new", [1, 2], ids=["rows", "chunks"])
def test_keys_of_the_lowest_value_count_nothing(max_new):
    """Scores that overflow to -infinity, against the same batch without these positions."""
    ensure_built()
    t, low = torch.bfloat16, torch.finfo(torch.bfloat16).min
    batch, part = (ref.Batch([(100, 2), (300, 2)], 1, 64, 16, t, seed=12) for _ in range(2))
    q = batch.randn(4, 16, 64).abs() + 0.1
    for b, pages in ((0, 6), (1, 11)):
        for p in range(16 * pages):
            at, slot = batch.place(b, p)
            batch.k[at, :, slot] = low
        part.table[b, :pages] = -1
    want, tol = ref.attention(part, q, 0.125, 0, torch.float32)
    assert float(tol.max()) < 0.05
    got = q8.attention(q8.PagedKV(*batch.cuda()), q.cuda(), max_new=max_new, dtype=torch.float32)
    device_ok()
    ref.close(got, want, tol)
