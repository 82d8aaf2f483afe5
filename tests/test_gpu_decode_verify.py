"""Decode == verify: what the norm, the MXFP4 product, the log probabilities and the decoder's end made
of them give for a token is bit for bit the same whether it comes alone or among up to 16 (the end: 15,
where its projection takes the GEMV)."""
import pytest
import torch

import ops_ref as ref
import q8_block_quantized_act_gb300 as q8
from gpu_util import device_ok, ensure_built
from q8_block_quantized_act_gb300 import score_tokens

pytestmark = pytest.mark.gpu
M = 16


def rnd(seed, *shape):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def spread(seed, rows, k):
    return rnd(seed, rows, k) * torch.exp(4 * rnd(seed + 1, rows, k // 32)).repeat_interleave(32, 1)


def bits(t):
    return t.contiguous().view(torch.int32 if t.element_size() == 4 else torch.int16)


@pytest.mark.parametrize("n,k", [(4096, 1792), (4096, 2048), (5120, 2560), (4096, 4096), (300, 8192), (1000, 512),
                                 (9226, 9984), (20481, 1280)])
def test_product(n, k):
    """Blocks of far-apart magnitudes: with like ones the f32 sums are exact in any order."""
    ensure_built()
    w, wsc = q8.quantize_mxfp4(spread(n, n, k))
    x = spread(k, M, k)
    alone = torch.cat([q8.gemm_mxfp4(w, wsc, x[t:t + 1]) for t in range(M)])
    device_ok()
    for m in range(1, M + 1):
        y = q8.gemm_mxfp4(w, wsc, x[:m])
        other = q8.gemm_mxfp4_preq(w, wsc, *q8.quantize_mxfp4(x[M - m:]))
        device_ok()
        assert torch.equal(bits(y), bits(alone[:m])), m
        assert torch.equal(bits(other), bits(alone[M - m:])), m


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("k", [256, 4096, 16640, 65536])
def test_norm(k, kind):
    ensure_built()
    x, r, w = (rnd(s, *shape).to(ref.TYPES[kind]) for s, shape in ((1, (M, k)), (2, (M, k)), (3, (k,))))
    y1 = torch.cat([q8.rmsnorm(x[t:t + 1], w, residual=r[t:t + 1]) for t in range(M)])
    for m in range(1, M + 1):
        y = torch.empty_like(x[:m])
        q, d = q8.rmsnorm_q8_1(x[:m], w, residual=r[:m], y=y)
        q1, d1 = q8.rmsnorm_q8_1(x[m - 1:m], w, residual=r[m - 1:m])
        device_ok()
        assert torch.equal(bits(y), bits(y1[:m])), m
        assert torch.equal(q[m - 1:], q1) and torch.equal(bits(d[m - 1:]), bits(d1)), m


@pytest.mark.parametrize("kind", ["f32", "f16"])
@pytest.mark.parametrize("v", [704, 8192, 50257, 128896])
def test_logprobs(v, kind):
    """Bit for bit where the rows start alike (modulo 16 bytes), the ids anyway."""
    ensure_built()
    x = (2.5 * rnd(v, M, v)).to(ref.TYPES[kind])
    tokens = torch.arange(M, device="cuda", dtype=torch.int32) * (v // M)
    parts = [q8.logprobs(x[t:t + 1].clone(), tokens[t:t + 1].clone(), top=5) for t in range(M)]
    alone = [torch.cat(p) for p in zip(*parts)]
    for m in range(1, M + 1):
        got = q8.logprobs(x[:m].clone(), tokens[:m].clone(), top=5)
        device_ok()
        assert torch.equal(got[2], alone[2][:m]), m
        if v % 8 == 0:
            for a, b in zip(got, alone):
                assert torch.equal(bits(a), bits(b[:m])), m


@pytest.mark.parametrize("k,vocab", [(512, 3004), (1792, 4096), (2560, 5120)])
def test_decoders_end(k, vocab):
    ensure_built()
    tail = score_tokens.make_tail(1 + 0.1 * rnd(1, k), 0.02 * rnd(2, k, k), 1 + 0.1 * rnd(3, k), 0.05 * spread(4, vocab, k))
    x, r = spread(5, M, k), rnd(6, M, k)
    tokens = torch.arange(M, device="cuda", dtype=torch.int32)
    parts = [score_tokens.score(tail, x[t:t + 1], r[t:t + 1].clone(), tokens[t:t + 1].clone(), top=4) for t in range(M)]
    alone = [torch.cat(p) for p in zip(*parts)]
    for m in range(1, q8.Q8ACT_GEMV_MAX_M + 1):
        got = score_tokens.score(tail, x[:m], r[:m].clone(), tokens[:m].clone(), top=4)
        device_ok()
        for a, b in zip(got, alone):
            assert torch.equal(bits(a), bits(b[:m])), m


def test_decoders_end_of_long_rows():
    """More tokens of a long row than the GEMV keeps at once."""
    ensure_built()
    k, vocab, m = 16384, 512, q8.Q8ACT_GEMV_MAX_M
    tail = score_tokens.make_tail(1 + 0.1 * rnd(1, k), 0.02 * rnd(2, k, k), 1 + 0.1 * rnd(3, k), 0.05 * rnd(4, vocab, k))
    x, r = rnd(5, m, k), rnd(6, m, k)
    tokens = torch.arange(m, device="cuda", dtype=torch.int32)
    parts = [score_tokens.score(tail, x[t:t + 1], r[t:t + 1].clone(), tokens[t:t + 1].clone(), top=4) for t in range(m)]
    got = score_tokens.score(tail, x, r.clone(), tokens, top=4)
    device_ok()
    for a, b in zip(got, (torch.cat(p) for p in zip(*parts))):
        assert torch.equal(bits(a), bits(b))
