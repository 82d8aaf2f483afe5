"""attention over a paged cache against the 64-bit form: decoding, a few tokens, chunks of prompts, mixed
batches; masks, places that do not exist, non-finite values in hidden places; graphs and streams."""
import math

import pytest
import torch

import paged_ref as ref
import q8_block_quantized_act_gb300 as q8
from gpu_util import device_ok, ensure_built

pytestmark = pytest.mark.gpu

# Rows of a unit that max_new announces: the kernels for up to 16 and 32 rows, whatever the batch holds, and the
# one for chunks.
HINTS = pytest.mark.parametrize("hint", [16, 32, 1000])


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def new(hint, q, hk):
    """max_new of so many rows (the call itself takes no more than there are)."""
    return max(1, hint * hk // q.shape[1])


def run(batch, q, hint, window=0, out_t=None, scale=None, out=None, ws=None):
    kv = q8.PagedKV(*batch.cuda())
    got = q8.attention(kv, q.cuda(), scale=scale, window=window, max_new=new(hint, q, batch.hk), dtype=out_t, out=out, ws=ws)
    device_ok()
    return got


def check(batch, hq, hint, window=0, out_t=None, scale=None, q=None, gain=1.0):
    q = gain * batch.randn(batch.m, hq, batch.d) if q is None else q
    out_t = out_t or batch.t
    want, tol = ref.attention(batch, q, scale or batch.d ** -0.5, window, out_t)
    out = torch.full(q.shape, 7.0, dtype=out_t, device="cuda")
    run(batch, q, hint, window, None, scale, out)
    mine = torch.zeros(batch.m, dtype=torch.bool)
    for r, _, _ in batch.tokens():
        mine[r] = True
    got = out.cpu()
    assert torch.equal(got[~mine], torch.full_like(got[~mine], 7.0))       # rows of no sequence
    ref.close(got[mine], want[mine], tol[mine])
    return got


LENGTHS = [
    [(0, 1)], [(15, 1), (16, 1), (14, 1)], [(62, 1), (63, 1), (64, 1), (126, 1), (127, 1), (128, 1)], [(1000, 1)],
    [(0, 5), (3, 0), (60, 3), (200, 1), (127, 2)],
    [(0, 40)], [(0, 127), (1, 130)], [(300, 70), (0, 1), (5, 0), (0, 260)],
]
HEADS = [(4, 4, 64, 16), (8, 2, 128, 64), (7, 1, 128, 16), (10, 2, 64, 32), (3, 1, 128, 128), (16, 1, 64, 256)]


@HINTS
@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("heads", HEADS, ids=str)
@pytest.mark.parametrize("seqs", LENGTHS, ids=str)
def test_lengths(seqs, heads, t, hint):
    hq, hk, d, page = heads
    check(ref.Batch(seqs, hk, d, page, ref.TYPES[t], seed=len(seqs)), hq, hint)


@HINTS
@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 100, 129, 1000])
def test_window(window, hint):
    batch = ref.Batch([(0, 150), (500, 3), (130, 1), (0, 1)], 2, 64, 16, torch.float16, seed=window)
    check(batch, 6, hint, window=window)


@HINTS
@pytest.mark.parametrize("out_t", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("t", ["f16", "bf16"])
def test_output_types_and_scale(t, out_t, hint):
    batch = ref.Batch([(33, 4), (200, 1), (0, 50)], 2, 128, 32, ref.TYPES[t], seed=4)
    check(batch, 4, hint, out_t=ref.TYPES[out_t], scale=0.3)


@HINTS
@pytest.mark.parametrize("hq,hk,d", [(40, 1, 64), (96, 2, 128), (300, 1, 64), (6, 6, 128)])
def test_groups_of_any_size(hq, hk, d, hint):
    """More query heads to a key head than a row tile has rows, and none to share with."""
    check(ref.Batch([(70, 3), (5, 1), (0, 20)], hk, d, 16, torch.float16, seed=hq), hq, hint)


@HINTS
def test_long_sequences_in_parts(hint):
    """Few rows over many positions: the sequence is shared by many CTAs and joined."""
    check(ref.Batch([(20000, 1)], 1, 128, 64, torch.bfloat16, seed=1), 4, hint)
    check(ref.Batch([(9000, 2), (40, 1), (5000, 1)], 2, 64, 16, torch.float16, seed=2), 6, hint)
    check(ref.Batch([(6000, 90)], 1, 64, 128, torch.float16, seed=3), 4, hint)


@pytest.mark.parametrize("window", [0, 260])
@pytest.mark.parametrize("seqs,heads", [
    ([(0, 600), (700, 300), (0, 0), (100, 450), (0, 900)], 8),
    ([(0, 500)] * 5, 16), ([(5000, 330), (0, 1), (40, 700), (2000, 128)], 16)], ids=["ragged", "even", "long"])
def test_more_units_than_ctas(seqs, heads, window):
    """Several chunks whose units the CTAs take longest first, some of them parts of row tiles; also none at all on one."""
    check(ref.Batch(seqs, heads, 64, 16, torch.float16, seed=heads), 2 * heads, 1000, window=window)


@HINTS
def test_many_sequences(hint):
    """More sequences than a CTA has threads, some without tokens."""
    seqs = [(i * 7 % 90, (1, 1, 0, 2)[i % 4]) for i in range(600)]
    check(ref.Batch(seqs, 1, 64, 16, torch.float16, seed=6), 2, hint)


@HINTS
@pytest.mark.parametrize("n,every", [(33, 13), (45, 13), (100, 13), (1100, 401)])
def test_parts_among_many_sequences(n, every, hint):
    """More than 32 sequences of which a few are long, so that some row tiles come in parts and most do not."""
    seqs = [(2500 + i, 5) if i % every == 2 else (i * 7 % 90, i % 3) for i in range(n)]
    check(ref.Batch(seqs, 2, 64, 16, torch.bfloat16, seed=n), 6, hint)
    check(ref.Batch(seqs, 2, 64, 16, torch.float16, seed=n), 8, hint, window=1500)


@HINTS
def test_padding_rows_are_left(hint):
    check(ref.Batch([(20, 3), (0, 2)], 2, 64, 16, torch.float16, seed=7, first=4, pad=9), 4, hint)


@HINTS
def test_rows_that_see_nothing(hint):
    """More new tokens than positions, a sequence of length 0, pages that do not exist at all."""
    batch = ref.Batch([(0, 6), (0, 2), (40, 2), (5, 1)], 2, 64, 16, torch.float16, seed=8)
    batch.lens[0] = 4
    batch.lens[1] = 0
    batch.table[2] = -1
    got = check(batch, 4, hint)
    assert float(got[:2].abs().max()) == 0.0 and float(got[6:10].abs().max()) == 0.0


@HINTS
def test_places_that_do_not_exist(hint):
    batch = ref.Batch([(200, 3), (90, 1), (64, 1), (0, 140)], 1, 128, 16, torch.bfloat16, seed=9)
    batch.table[0, 3] = -1
    batch.table[0, 12] = batch.pages
    batch.table[1, 0] = -2 ** 31
    batch.table[3, 2] = 2 ** 31 - 1
    batch.table = batch.table[:, :13].contiguous()
    batch.width = 13
    batch.lens[2] = 2 ** 31 - 1                     # a length beyond the table
    batch.seqs[2] = (2 ** 31 - 2, 1)
    q = batch.randn(batch.m, 4, 128)
    short = ref.Batch([(200, 3), (90, 1), (207, 1), (0, 140)], 1, 128, 16, torch.bfloat16, seed=9)
    short.k, short.v, short.table, short.width, short.pages = batch.k, batch.v, batch.table, 13, batch.pages
    want, tol = ref.attention(short, q, 128 ** -0.5, 0, batch.t)
    ref.close(run(batch, q, hint), want, tol)


@HINTS
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("t", ["f16", "bf16"])
def test_hidden_values_do_not_matter(bad, t, hint):
    """Non-finite keys and values at later positions, behind the window and beyond lens."""
    t = ref.TYPES[t]
    batch = ref.Batch([(60, 9), (0, 150)], 1, 64, 16, t, seed=10, filler=bad)
    for b, p in ((0, 66), (1, 70), (1, 149)):       # seen by the tokens from there on only
        at, slot = batch.place(b, p)
        batch.v[at, :, slot, 3] = bad
    q = batch.randn(batch.m, 2, 64)
    for window in (0, 20):
        want, tol = ref.attention(batch, q, 0.125, window, t)
        ref.close(run(batch, q, hint, window), want, tol)
    # keys: a score of NaN spoils the rows that see it and no others
    for b, p in ((0, 66), (1, 70)):
        at, slot = batch.place(b, p)
        batch.k[at, :, slot, 5] = math.nan
    got = run(batch, q, hint, 0).cpu()
    for r, b, p in batch.tokens():
        assert bool(torch.isnan(got[r]).all()) == (p >= (66, 70)[b]), (b, p)


@HINTS
@pytest.mark.parametrize("d", [64, 128])
def test_hidden_values_in_long_sequences(d, hint):
    """The same where several CTAs, and both halves of one, have parts of a row: values in tiles of either half."""
    t = torch.float16
    batch = ref.Batch([(1500, 9), (2430, 3)], 1, d, 32, t, seed=19, filler=math.nan)
    for b, p in ((0, 1503), (0, 1507), (1, 2431), (1, 2432)):
        at, slot = batch.place(b, p)
        batch.v[at, :, slot, 3] = math.inf
    q = batch.randn(batch.m, 3, d)
    for window in (0, 1300):
        want, tol = ref.attention(batch, q, d ** -0.5, window, t)
        ref.close(run(batch, q, hint, window), want, tol)


@HINTS
def test_non_finite_value_in_many_long_sequences(hint):
    """Units of whole long sequences (there are too many to cut), whose newest value is an infinity: every sequence is the
    first one again."""
    one = ref.Batch([(9000, 3)], 1, 128, 64, torch.bfloat16, seed=20)
    at, slot = one.place(0, 9001)
    one.v[at, 0, slot, 7] = math.inf
    one.v[at, 0, slot, 70] = math.nan
    n, q = 500, one.randn(3, 2, 128)
    want, tol = ref.attention(one, q, 128 ** -0.5, 0, one.t)
    kd, vd, table, _, _ = one.cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    kv = q8.PagedKV(kd, vd, table.expand(n, -1).contiguous(), 3 * torch.arange(n + 1, **i32), torch.full((n,), 9003, **i32))
    got = q8.attention(kv, q.cuda().repeat(n, 1, 1), max_new=new(hint, q, 1)).view(n, 3, 2, 128)
    device_ok()
    ref.close(got, want.expand(n, -1, -1, -1), tol.expand(n, -1, -1, -1))


@HINTS
def test_lowest_values_and_large_scores(hint):
    """Scores that overflow to -inf count nothing, large ones pick one position."""
    batch = ref.Batch([(100, 2), (0, 30)], 1, 64, 16, torch.float16, seed=11)
    check(batch, 2, hint, gain=30.0)
    t = torch.bfloat16
    batch = ref.Batch([(100, 2)], 1, 64, 16, t, seed=12)
    low = torch.finfo(t).min
    for p in range(0, 90):
        at, slot = batch.place(0, p)
        batch.k[at, :, slot] = low
    q = batch.randn(2, 2, 64).abs() + 0.1
    got = run(batch, q, hint).cpu().double()
    part = ref.Batch([(100, 2)], 1, 64, 16, t, seed=12)
    w, tol = ref.attention(batch, q, 0.125, 0, t)
    keep = torch.isfinite(w)
    assert torch.isfinite(got).all()
    ref.close(got[keep], w[keep], tol[keep])


@HINTS
def test_rising_scores(hint):
    """Every position scores above all before it: the running maximum moves at each tile."""
    batch = ref.Batch([(700, 1), (300, 140)], 1, 64, 16, torch.float16, seed=13)
    for b, (c, n) in enumerate(batch.seqs):
        for p in range(c + n):
            at, slot = batch.place(b, p)
            batch.k[at, :, slot] = p / 16.0
    q = torch.full((batch.m, 2, 64), 0.25, dtype=torch.float16)
    check(batch, 2, hint, q=q)


@HINTS
def test_strided_arguments(hint):
    """q and out as parts of wider rows, table rows apart, k and v as halves of one tensor."""
    batch = ref.Batch([(50, 3), (7, 1), (0, 66)], 2, 64, 16, torch.float16, seed=14)
    m = batch.m
    wide = batch.randn(m, 9, 64)
    q = wide[:, 2:6]
    want, tol = ref.attention(batch, q, 0.125, 0, torch.float32)
    both = torch.stack((batch.k, batch.v), 1).cuda()
    table = torch.full((3, batch.width + 5), 2 ** 30, dtype=torch.int32, device="cuda")
    table[:, :batch.width] = batch.table.cuda()
    kv = q8.PagedKV(both[:, 0], both[:, 1], table[:, :batch.width], batch.starts.cuda(), batch.lens.cuda())
    out = torch.full((m, 6, 64), 7.0, device="cuda")
    q8.attention(kv, wide.cuda()[:, 2:6], out=out[:, 1:5], max_new=new(hint, q, 2))
    device_ok()
    ref.close(out[:, 1:5], want, tol)
    assert bool((out[:, 0] == 7).all()) and bool((out[:, 5] == 7).all())


@HINTS
def test_same_bits_each_time(hint):
    batch = ref.Batch([(3000, 1), (500, 40), (0, 200)], 2, 128, 16, torch.bfloat16, seed=15)
    q = batch.randn(batch.m, 8, 128)
    a = run(batch, q, hint)
    for _ in range(3):
        assert torch.equal(a.view(torch.int16), run(batch, q, hint).view(torch.int16))


@HINTS
def test_graph_follows_lengths(hint):
    """One captured call, replayed while the sequences grow and change pages."""
    hk, hq, d, page = 1, 4, 64, 16
    batch = ref.Batch([(2990, 1), (70, 3), (0, 1)], hk, d, page, torch.float16, seed=16)
    kd, vd, table, starts, lens = batch.cuda()
    kv = q8.PagedKV(kd, vd, table, starts, lens)
    q = batch.randn(5, hq, d)
    qd, out, ws = q.cuda(), torch.empty((5, hq, d), dtype=torch.float16, device="cuda"), q8.attention_workspace(kv, hq)
    q8.attention(kv, qd, max_new=new(hint, q, hk), ws=ws, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q8.attention(kv, qd, max_new=new(hint, q, hk), ws=ws, out=out)
    for n in ([1, 3, 1], [2991, 73, 1], [100, 20, 0], [2000, 5, 1]):
        batch.lens = torch.tensor(n, dtype=torch.int32)
        lens.copy_(batch.lens)
        out.fill_(7.0)
        g.replay()
        device_ok()
        want, tol = ref.attention(batch, q, 0.125, 0, torch.float16)
        ref.close(out, want, tol)


@HINTS
def test_two_graphs_share_a_workspace(hint):
    """Replayed in turn on one stream, over different batches."""
    ws, graphs = None, []
    for seed, seqs in ((21, [(2000, 1), (90, 3)]), (22, [(0, 150), (700, 2), (3000, 1)])):
        batch = ref.Batch(seqs, 2, 64, 16, torch.float16, seed=seed)
        q = batch.randn(batch.m, 4, 64)
        kv, qd = q8.PagedKV(*batch.cuda()), q.cuda()
        ws = q8.attention_workspace(kv, 4) if ws is None else ws
        out = torch.empty_like(qd)
        call = lambda: q8.attention(kv, qd, max_new=new(hint, q, 2), ws=ws, out=out)     # noqa: B023, E731
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append((g, kv, qd, out, ref.attention(batch, q, 0.125, 0, torch.float16)))
    for _ in range(3):
        for g, _, _, out, _ in graphs:
            out.fill_(7.0)
            g.replay()
    device_ok()
    for _, _, _, out, (want, tol) in graphs:
        ref.close(out, want, tol)


def test_two_streams():
    """Two calls at once, with a workspace each."""
    batch = ref.Batch([(4000, 1), (900, 2)], 2, 64, 16, torch.float16, seed=17)
    q = batch.randn(3, 4, 64)
    kv = q8.PagedKV(*batch.cuda())
    qd = q.cuda()
    want, tol = ref.attention(batch, q, 0.125, 0, torch.float16)
    torch.cuda.synchronize()
    outs = []
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [q8.attention_workspace(kv, 4) for _ in streams]
    for i in range(6):
        with torch.cuda.stream(streams[i % 2]):
            outs.append(q8.attention(kv, qd, max_new=2, ws=spaces[i % 2]))
    device_ok()
    for o in outs:
        ref.close(o, want, tol)


@HINTS
def test_shared_pages(hint):
    """Two sequences with a common beginning on the same pages, and one sequence twice in the batch."""
    batch = ref.Batch([(60, 2), (60, 2), (60, 2)], 1, 64, 16, torch.float16, seed=18)
    batch.table[1, :3] = batch.table[0, :3]
    batch.table[2] = batch.table[0]
    check(batch, 2, hint)
