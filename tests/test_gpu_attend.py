"""The attention block as it is used: norm -> Q8_0 projection -> rotation and append -> attention -> Q8_0 projection."""
import pytest
import torch

import paged_ref as ref
import q8_block_quantized_act_gb300 as q8
from gpu_util import device_ok, ensure_built
from q8_block_quantized_act_gb300 import attend

pytestmark = pytest.mark.gpu
K, HQ, HK, D, PAGE = 512, 8, 2, 64, 16


def block(seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")   # noqa: E731
    return attend.make_block(1 + 0.1 * rnd(K), 0.05 * rnd((HQ + 2 * HK) * D, K), 0.05 * rnd(K, HQ * D), HQ, HK, D), rnd


def paged(seqs, t=torch.float16, seed=0):
    batch = ref.Batch(seqs, HK, D, PAGE, t, seed=seed, filler=0.0)
    return batch, q8.PagedKV(*batch.cuda())


def same(a, b):
    return torch.equal(a.view(torch.int32), b.view(torch.int32))


@pytest.mark.parametrize("seqs", [[(5, 1)], [(40, 3), (0, 2), (17, 1)], [(0, 40)], [(30, 9), (100, 1), (0, 25)]], ids=str)
def test_block_follows_its_parts(seqs):
    """Append and attention against the 64-bit forms of these stages on the GPU's own inputs of them; the other
    stages, and the whole on a side stream, bit for bit."""
    ensure_built()
    b, rnd = block()
    batch, kv = paged(seqs)
    m = batch.m
    x, r = rnd(m, K), rnd(m, K)
    r1 = r.clone()
    got = attend.attend(b, kv, x, r1)
    device_ok()

    n = (HQ + 2 * HK) * D
    s = torch.empty_like(r)
    if m <= 15:
        y = q8.gemv_q8_0(b.qkv, *q8.rmsnorm_q8_1(x, b.norm, residual=r, residual_out=s), n)
    else:
        y = q8.gemm_q8_0_preq(b.qkv, *q8.rmsnorm_q8_1_mmq(x, b.norm, residual=r, residual_out=s), n)
    assert torch.equal(s, r1)
    y = y.view(m, HQ + 2 * HK, D)
    host = y.cpu()
    freqs = [10000.0 ** (-2 * i / D) for i in range(D // 2)]
    (q64, qtol), (k64, ktol), vc = ref.append(batch, host[:, :HQ], host[:, HQ:HQ + HK], host[:, HQ + HK:], freqs, False, batch.t)
    wrote = ~torch.isnan(k64)
    ref.close(kv.k.cpu()[wrote], k64[wrote], ktol[wrote], "k")
    assert torch.equal(kv.v.cpu(), vc)
    q = q8.append_kv(kv, y[:, :HQ], y[:, HQ:HQ + HK], y[:, HQ + HK:], turns=b.turns)
    ref.close(q, q64, qtol, "q")
    batch.k, batch.v = kv.k.cpu(), kv.v.cpu()
    want, tol = ref.attention(batch, q.cpu(), D ** -0.5, 0, torch.float32)
    o = q8.attention(kv, q, dtype=torch.float32)
    ref.close(o, want, tol, "attention")
    o = o.view(m, HQ * D)
    h = q8.gemv_q8_0(b.out, *q8.quantize_q8_1(o), K) if m <= 15 else q8.gemm_q8_0(b.out, o, K)
    device_ok()
    assert same(h, got)

    side = torch.cuda.Stream()
    _, kv2 = paged(seqs)
    r2 = r.clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        again = attend.attend(b, kv2, x, r2)
    device_ok()
    assert same(again, got) and torch.equal(kv2.k, kv.k)


def test_decoding_by_a_captured_graph():
    """A step captured once and replayed while two sequences grow over page borders: the eager calls' bits."""
    ensure_built()
    b, rnd = block(1)
    steps = 40
    xs = rnd(steps, 2, K)

    def start():
        batch, kv = paged([(0, 1), (0, 1)], seed=3)
        pages = torch.arange(2 * 4, dtype=torch.int32).view(2, 4)
        k, v = (torch.zeros((8, HK, PAGE, D), dtype=torch.float16, device="cuda") for _ in range(2))
        lens = torch.tensor([0, 9], dtype=torch.int32, device="cuda")
        return q8.PagedKV(k, v, pages.cuda(), kv.starts, lens)

    eager, kv = [], start()
    for x in xs:
        kv.lens += 1
        eager.append(attend.attend(b, kv, x, torch.zeros_like(x), max_new=1))
    kv = start()
    x, r, ws = xs[0].clone(), torch.zeros((2, K), device="cuda"), q8.attention_workspace(kv, HQ)
    kv.lens += 1
    attend.attend(b, kv, x, r, max_new=1, ws=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        h = attend.attend(b, kv, x, r, max_new=1, ws=ws)
    kv.lens -= 1
    for i in range(steps):
        x.copy_(xs[i])
        r.zero_()
        kv.lens += 1
        g.replay()
        torch.cuda.synchronize()
        assert same(h, eager[i]), i
    device_ok()


def test_command_runs(capsys):
    ensure_built()
    attend.main(["--prompt", "50", "--steps", "3", "--k", "512"])
    assert "decoded one by one: 3 tokens" in capsys.readouterr().out
