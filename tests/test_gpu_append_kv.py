"""append_kv: rotation of queries and keys, keys and values into the pages, against the 64-bit form."""
import math

import pytest
import torch

import paged_ref as ref
import q8_block_quantized_act_gb300 as q8
from gpu_util import device_ok, ensure_built

pytestmark = pytest.mark.gpu
BASE = 500000.0


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def freqs(rot, scale=1.0):
    return [scale * BASE ** (-2 * i / rot) for i in range(rot // 2)]


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


def check(batch, hq, src, rot, interleaved, fused=True):
    t, hk, d, m = batch.t, batch.hk, batch.d, batch.m
    f = freqs(rot) if rot else []
    qkv = batch.randn(m, hq + 2 * hk, d, t=src)
    if not fused:
        q, k, v = qkv[:, :hq].contiguous(), qkv[:, hq:hq + hk].contiguous(), qkv[:, hq + hk:].contiguous()
    else:
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    (q64, qtol), (k64, ktol), vc = ref.append(batch, q, k, v, f, interleaved, t)
    kd, vd, table, starts, lens = batch.cuda()
    kv = q8.PagedKV(kd, vd, table, starts, lens)
    dev = qkv.cuda()
    parts = (dev[:, :hq], dev[:, hq:hq + hk], dev[:, hq + hk:])
    if not fused:
        parts = [x.contiguous() for x in parts]
    out = torch.full((m, hq, d), 7.0, dtype=t, device="cuda")
    turns = q8.rope_turns(f, "cuda") if f else None
    got = q8.append_kv(kv, *parts, turns=turns, interleaved=interleaved, out=out)
    assert got is out
    device_ok()
    mine = ~torch.isnan(q64)
    gq = out.cpu()
    assert torch.equal(gq[~mine], torch.full_like(gq[~mine], 7.0))              # rows behind the last sequence
    ref.close(gq[mine], q64[mine], qtol[mine], "q")
    wrote = ~torch.isnan(k64)
    gk = kd.cpu()
    ref.close(gk[wrote], k64[wrote], ktol[wrote], "k")
    assert same_bits(gk[~wrote], batch.k[~wrote])
    assert same_bits(vd.cpu(), vc)


SEQS = [
    [(0, 1)], [(4095, 1)], [(5, 1), (0, 1), (63, 1), (64, 1)],
    [(3, 7), (0, 0), (100, 1), (0, 33), (17, 0)],
]


@pytest.mark.parametrize("src", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("hq,hk,d,rot,page", [(4, 2, 64, 64, 16), (8, 1, 128, 128, 64), (3, 3, 128, 32, 32), (7, 1, 64, 48, 16),
                                              (2, 1, 128, 0, 128)])
def test_types_and_heads(src, t, interleaved, hq, hk, d, rot, page):
    for i, seqs in enumerate(SEQS):
        batch = ref.Batch(seqs, hk, d, page, ref.TYPES[t], seed=i, pad=i % 2)
        check(batch, hq, ref.TYPES[src], rot, interleaved, fused=i != 1)


@pytest.mark.parametrize("hq,hk,d", [(32, 8, 128), (12, 12, 64)])
def test_many_tokens(hq, hk, d):
    """The variant with several tokens a CTA, ragged, with padding before and behind."""
    batch = ref.Batch([(9, 1211), (100, 1), (0, 0), (0, 1300)], hk, d, 16, torch.bfloat16, seed=3, first=2, pad=3)
    check(batch, hq, torch.bfloat16, d, False)


def test_far_positions():
    """Angles of positions near 2^30, where f32 (and a product in it) would have lost the turn."""
    d, page = 128, 1024
    f = freqs(d)
    x = torch.randn((3, 3, d), generator=torch.Generator().manual_seed(5))
    ends = [2 ** 30, 2 ** 30 - 1000, 123456789]
    width = 2 ** 30 // page
    table = torch.full((3, width), -1, dtype=torch.int32)
    for b, n in enumerate(ends):
        table[b, (n - 1) // page] = b
    kc = torch.zeros((3, 1, page, d), dtype=torch.float16, device="cuda")
    kv = q8.PagedKV(kc, kc.clone(), table.cuda(), torch.arange(4, dtype=torch.int32, device="cuda"),
                    torch.tensor(ends, dtype=torch.int32, device="cuda"))
    xd = x.cuda()
    got = q8.append_kv(kv, xd[:, :1], xd[:, 1:2], xd[:, 2:], turns=q8.rope_turns(f, "cuda"))
    device_ok()
    pos = torch.tensor(ends, dtype=torch.float64) - 1
    # the 64-bit reference's own angle: 2^30 * 2^-53 of f in radians
    own = 2.0 ** 30 * 2.0 ** -52
    want, size = ref.rotated(x.double(), pos, f, False)
    tol = (ref.ROTATION + own) * size + ref.half(torch.float16) * want.abs() + ref.tiny(torch.float16)
    ref.close(got[:, 0], want[:, 0], tol[:, 0], "q")
    for b, n in enumerate(ends):
        ref.close(kc[b, 0, (n - 1) % page], want[b, 1], tol[b, 1], "k")


def test_places_that_do_not_exist():
    """Pages outside the cache, positions beyond the table and before 0: nothing is written."""
    batch = ref.Batch([(10, 20), (40, 9), (0, 5), (2, 3)], 2, 64, 16, torch.float16, seed=1, filler=3.0)
    batch.table[0, 1] = -1
    batch.table[1, 2] = batch.pages                     # one beyond the last
    batch.table[3, 0] = 2 ** 31 - 1
    batch.lens[2] = 2                                   # five tokens for two positions
    batch.width = 3
    batch.table = batch.table[:, :3].contiguous()       # the last positions of sequence 1 lie behind it
    check(batch, 4, torch.float32, 64, False)


def test_in_place_and_without_queries():
    batch = ref.Batch([(30, 5), (1, 2)], 2, 128, 16, torch.bfloat16, seed=2)
    q, k, v = batch.randn(7, 6, 128), batch.randn(7, 2, 128), batch.randn(7, 2, 128)
    f = freqs(128)
    (q64, qtol), (k64, ktol), vc = ref.append(batch, q, k, v, f, False, batch.t)
    kd, vd, *rest = batch.cuda()
    kv = q8.PagedKV(kd, vd, *rest)
    qd = q.cuda()
    turns = q8.rope_turns(f, "cuda")
    assert q8.append_kv(kv, None, k.cuda(), v.cuda(), turns=turns) is None
    wrote = ~torch.isnan(k64)
    ref.close(kd.cpu()[wrote], k64[wrote], ktol[wrote], "k")
    q8.append_kv(kv, qd, k.cuda(), v.cuda(), turns=turns, out=qd)
    device_ok()
    ref.close(qd, q64, qtol, "q")
    assert same_bits(vd.cpu(), vc)


def test_pages_apart_and_graph():
    """k and v as halves of one tensor; a captured call follows lens and table."""
    hk, d, page, pages = 2, 64, 16, 9
    both = torch.zeros((pages, 2, hk, page, d), dtype=torch.float16, device="cuda")
    table = torch.tensor([[0, 4], [7, 2]], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    lens = torch.tensor([1, 1], dtype=torch.int32, device="cuda")
    kv = q8.PagedKV(both[:, 0], both[:, 1], table, starts, lens)
    x = torch.randn((2, 6, d), device="cuda")
    args = (x[:, :2], x[:, 2:4], x[:, 4:])
    turns = q8.rope_turns(freqs(d), "cuda")
    out = torch.empty((2, 2, d), dtype=torch.float16, device="cuda")
    q8.append_kv(kv, *args, turns=turns, out=out)
    torch.cuda.synchronize()
    both.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q8.append_kv(kv, *args, turns=turns, out=out)
    for step in range(1, 20):
        lens.fill_(step)
        g.replay()
    device_ok()
    host = both.cpu()
    for b, row in enumerate(table.tolist()):
        for p in range(19):
            want, size = ref.rotated(x[b:b + 1, 2:4].cpu().double(), torch.tensor([float(p)], dtype=torch.float64), freqs(d), False)
            ref.close(host[row[p // page], 0, :, p % page], want[0],
                      ref.ROTATION * size[0] + ref.half(torch.float16) * want[0].abs() + ref.tiny(torch.float16), "k")
            assert torch.equal(host[row[p // page], 1, :, p % page], x[b, 4:].cpu().half())
    assert float(host[[1, 3, 5, 6, 8]].abs().max()) == 0.0


def test_rope_turns():
    t = q8.rope_turns([2 * math.pi / 4, 1.0, 0.0, -1.0], "cuda")
    assert t.dtype is torch.int64 and t[0].item() == 2 ** 62 and t[2].item() == 0 and t[3].item() == -t[1].item()
