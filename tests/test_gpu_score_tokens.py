"""The decoder's end as it is used: norm -> Q8_0 projection -> norm -> MXFP4 head -> log probabilities."""
import numpy as np
import pytest
import torch

import ops_ref as ref
import q8_block_quantized_act_gb300 as q8
from gpu_util import device_ok, ensure_built, host
from q8_block_quantized_act_gb300 import score_tokens

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m", [1, 7, 15, 16, 40])
def test_score_follows_its_parts(m):
    """Each stage against the 64-bit form of that stage on the GPU's own inputs of it, and the whole
    again on a side stream, bit for bit."""
    ensure_built()
    k, vocab, top = 512, 3001, 6
    g = torch.Generator(device="cuda").manual_seed(m)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")   # noqa: E731
    w1, proj, w2, head = 1 + 0.1 * rnd(k), 0.02 * rnd(k, k), 1 + 0.1 * rnd(k), 0.05 * rnd(vocab, k)
    x, r = rnd(m, k), rnd(m, k)
    tokens = torch.randint(0, vocab, (m,), generator=g, device="cuda").to(torch.int32)
    tail = score_tokens.make_tail(w1, proj, w2, head)

    r1 = r.clone()
    got = score_tokens.score(tail, x, r1, tokens, top=top)
    device_ok()

    # the stages on their own
    s = torch.empty_like(r)
    xq, xd = q8.rmsnorm_q8_1(x, w1, residual=r, residual_out=s)
    if m <= 15:
        h = q8.gemv_q8_0(tail.proj, xq, xd, k)
    else:
        qh, dt = q8.rmsnorm_q8_1_mmq(x, w1, residual=r)
        h = q8.gemm_q8_0_preq(tail.proj, qh, dt, k)
    s2 = torch.empty_like(r)
    y = q8.rmsnorm(h, w2, residual=s, residual_out=s2)
    yq = torch.empty_like(y)
    q8.rmsnorm_q8_1(h, w2, residual=s, y=yq)
    logits = q8.gemm_mxfp4(tail.head, tail.head_scales, y)
    device_ok()
    assert torch.equal(yq, y)                      # the norm alone is the quantizing norm's y
    s_ref, y64 = ref.rmsnorm(h.cpu(), s.cpu(), w2.cpu(), 1e-6)
    assert torch.equal(s2.cpu(), s_ref) and torch.equal(r1, s2)
    assert np.all(np.abs(ref.f64(y) - y64) <= ((k / 64 + 32) / 2 + 9) * ref.U * np.abs(y64))
    yb, yc = ref.mxfp4_quantize(ref.f64(y))
    hb, hc = ref.mxfp4_quantize(ref.f64(head))
    yv, hv = ref.mxfp4_values(yb, yc), ref.mxfp4_values(hb, hc)
    assert np.all(np.abs(ref.f64(logits) - yv @ hv.T) <= 1e-5 * (np.abs(yv) @ np.abs(hv).T))
    lp, ent, ids, tlp = ref.logprobs(ref.f64(logits), tokens.cpu().numpy(), top)
    assert np.array_equal(host(got[2]), ids)
    tol = (vocab / 512 + 40) * ref.U + 2.0 ** -22 * (1 + np.log(vocab) + np.abs(lp))
    assert np.all(np.abs(host(got[0]) - lp) <= tol)
    assert np.all(np.abs(host(got[3]) - tlp) <= tol[:, None] + 2.0 ** -22 * np.abs(tlp))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        r2 = r * 1.0
        again = score_tokens.score(tail, x * 1.0, r2, tokens, top=top)
    side.synchronize()
    device_ok()
    for a, b in zip(got, again):
        assert torch.equal(a, b)


def test_score_in_a_cuda_graph():
    """The five calls captured once and replayed on new hidden states."""
    ensure_built()
    m, k, vocab = 3, 512, 2000
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")   # noqa: E731
    tail = score_tokens.make_tail(1 + 0.1 * rnd(k), 0.02 * rnd(k, k), 1 + 0.1 * rnd(k), 0.05 * rnd(vocab, k))
    tokens = torch.arange(m, device="cuda", dtype=torch.int32)
    sets = [(rnd(m, k), rnd(m, k)) for _ in range(3)]
    want = [score_tokens.score(tail, x, r.clone(), tokens, top=4) for x, r in sets]
    x, r = torch.zeros((m, k), device="cuda"), torch.zeros((m, k), device="cuda")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        score_tokens.score(tail, x, r, tokens, top=4)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = score_tokens.score(tail, x, r, tokens, top=4)
    torch.cuda.synchronize()
    for (xi, ri), w in zip(sets, want):
        x.copy_(xi)
        r.copy_(ri)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, w):
            assert torch.equal(a, b)
    device_ok()


def test_score_command(capsys):
    ensure_built()
    score_tokens.main(["--m", "20", "--k", "512", "--vocab", "1000", "--top", "3"])
    out = capsys.readouterr().out
    assert "20 tokens, mean log p -" in out
