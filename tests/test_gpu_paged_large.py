"""A cache of more than 2^32 elements, strides that pass 32 bits, many sequences: the places that matter are
far apart, the values as in a small cache."""
import pytest
import torch

import paged_ref as ref
import q8_block_quantized_act_gb300 as q8
from gpu_util import device_ok, ensure_built

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hint", [1, None])
@pytest.mark.parametrize("apart", [False, True], ids=["pages adjacent", "pages far apart"])
def test_cache_past_32_bits(apart, hint):
    ensure_built()
    t, hk, d, page = torch.bfloat16, 2, 128, 16
    batch = ref.Batch([(37, 30), (20, 1)], hk, d, page, t, seed=1, filler=0.0, spare=0)
    hq, m = 6, batch.m
    q, k, v = (batch.randn(m, h, d) for h in (hq, hk, hk))
    inv = [10000.0 ** (-2 * i / d) for i in range(d // 2)]
    (q64, qtol), (k64, ktol), vc = ref.append(batch, q, k, v, inv, False, t)
    size = hk * page * d
    if apart:
        gap = 2 ** 32 // (batch.pages - 2) // size + 1                    # pages apart, so that the last is past 2^32
        many, at = (batch.pages - 1) * gap + 1, torch.arange(batch.pages) * gap
        big = [torch.zeros((many, hk, page, d), dtype=t, device="cuda") for _ in range(2)]
        caches = [c[::gap] for c in big]
        table = batch.table
    else:
        many = 2 ** 32 // size + 5
        at = many - batch.pages + torch.arange(batch.pages)
        big = [torch.zeros((many, hk, page, d), dtype=t, device="cuda") for _ in range(2)]
        caches = big
        table = torch.where(batch.table >= 0, batch.table + (many - batch.pages), batch.table)
    for c, src in zip(big, (batch.k, batch.v)):
        c[at.cuda()] = src.cuda()
    kv = q8.PagedKV(*caches, table.cuda(), batch.starts.cuda(), batch.lens.cuda())
    got = q8.append_kv(kv, q.cuda(), k.cuda(), v.cuda(), turns=q8.rope_turns(inv, "cuda"))
    o = q8.attention(kv, got, max_new=hint)
    device_ok()
    ref.close(got, q64, qtol, "q")
    kd, vd = big[0][at.cuda()].cpu(), big[1][at.cuda()].cpu()
    wrote = ~torch.isnan(k64)
    ref.close(kd[wrote], k64[wrote], ktol[wrote], "k")
    assert torch.equal(vd, vc)
    batch.k, batch.v = kd, vd
    want, tol = ref.attention(batch, got.cpu(), d ** -0.5, 0, t)
    ref.close(o, want, tol)
    for c in big:
        c[at.cuda()] = 0
        assert not c.any()


def test_rows_far_apart():
    """Tokens of q, k, v and out farther apart than 2^31 elements in all."""
    ensure_built()
    t, hk, d, page, m = torch.float16, 1, 64, 16, 3
    batch = ref.Batch([(30, 3)], hk, d, page, t, seed=2)
    ld = 2 ** 30 + 8
    wide = torch.empty(2 * ld + 4 * d, dtype=t, device="cuda").as_strided((m, 4, d), (ld, d, 1))
    x = batch.randn(m, 4, d)
    wide.copy_(x.cuda())
    (q64, qtol), (k64, ktol), vc = ref.append(batch, x[:, :2], x[:, 2:3], x[:, 3:], [1.0, 0.1] * 16, True, t)
    kv = q8.PagedKV(*batch.cuda())
    q8.append_kv(kv, wide[:, :2], wide[:, 2:3], wide[:, 3:], turns=q8.rope_turns([1.0, 0.1] * 16, "cuda"), interleaved=True,
                 out=wide[:, :2])
    device_ok()
    ref.close(wide[:, :2], q64, qtol, "q")
    wrote = ~torch.isnan(k64)
    ref.close(kv.k.cpu()[wrote], k64[wrote], ktol[wrote], "k")
    batch.k, batch.v, q = kv.k.cpu(), kv.v.cpu(), wide[:, :2].cpu()
    want, tol = ref.attention(batch, q, 0.125, 0, t)
    for hint in (1, None):
        q8.attention(kv, wide[:, :2], max_new=hint, out=wide[:, 2:])
        device_ok()
        ref.close(wide[:, 2:], want, tol)


@pytest.mark.parametrize("hint", [1, 1000])
def test_thousands_of_sequences(hint):
    """More sequences than threads or lanes count one by one, of every length, some empty."""
    ensure_built()
    seqs = [(i * 7 % 40, (1, 0, 1, 3, 1)[i % 5]) for i in range(1300)]
    batch = ref.Batch(seqs, 1, 64, 16, torch.float16, seed=4)
    q = batch.randn(batch.m, 2, 64)
    want, tol = ref.attention(batch, q, 0.125, 0, torch.float16)
    out = q8.attention(q8.PagedKV(*batch.cuda()), q.cuda(), max_new=hint)
    device_ok()
    ref.close(out, want, tol)
