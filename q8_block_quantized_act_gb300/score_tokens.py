"""The end of a decoder: a block-quantized projection, the head and the tokens' log probabilities.

    python -m q8_block_quantized_act_gb300.score_tokens --m 5 --k 4096 --vocab 64448

For m hidden states x and their residual stream:

    residual += x; norm; q8_1          rmsnorm_q8_1 (m <= 15) or rmsnorm_q8_1_mmq
    h = projection (Q8_0 x q8_1)       gemv_q8_0 (m <= 15) or gemm_q8_0_preq
    residual += h; norm                rmsnorm
    logits = head (MXFP4)              gemm_mxfp4
    log probabilities, entropy, top    logprobs

five calls on one stream, no host synchronization between them.  The command draws synthetic hidden
states and weights, scores random tokens and prints what a caller would look at.
"""
from __future__ import annotations

import argparse
from dataclasses import dataclass

import q8_block_quantized_act_gb300 as q8


@dataclass
class Tail:
    """Weights of the decoder's end: two norms, a Q8_0 projection [k, k], an MXFP4 head [vocab, k]."""
    norm1: object
    proj: object          # Q8_0 bytes
    norm2: object
    head: object          # MXFP4 codes
    head_scales: object   # tiled scales


def make_tail(norm1, proj, norm2, head) -> Tail:
    """Quantize float32 CUDA weights once, at load time."""
    codes, scales = q8.quantize_mxfp4(head)
    return Tail(norm1, q8.quantize_q8_0(proj), norm2, codes, scales)


def project(w, xq, xd, n: int, out):
    """The GEMV of up to Q8ACT_GEMV_MAX_M tokens for any k: it keeps the whole activation in shared memory
    and refuses what does not fit, so long rows go through it in parts (a token's bits do not depend on
    how many it comes with)."""
    m = xq.shape[0]
    try:
        return q8.gemv_q8_0(w, xq, xd, n, out=out)
    except q8.Q8ActError as e:
        if e.rc != q8.Q8ACT_ERR_DIMS or m == 1:
            raise
    project(w, xq[:m // 2], xd[:m // 2], n, out[:m // 2])
    project(w, xq[m // 2:], xd[m // 2:], n, out[m // 2:])
    return out


def score(tail: Tail, x, residual, tokens, top: int = 0, eps: float = 1e-6):
    """x, residual [m, k] float32 (the residual stream is updated in place), tokens [m] int32 ->
    (logprob [m], entropy [m], top ids, top log probabilities)."""
    m, k = x.shape
    if m <= q8.Q8ACT_GEMV_MAX_M:
        xq, xd = q8.rmsnorm_q8_1(x, tail.norm1, eps, residual=residual, residual_out=residual)
        h = project(tail.proj, xq, xd, k, x.new_empty((m, k)))
    else:
        xqh, xdt = q8.rmsnorm_q8_1_mmq(x, tail.norm1, eps, residual=residual, residual_out=residual)
        h = q8.gemm_q8_0_preq(tail.proj, xqh, xdt, k)
    y = q8.rmsnorm(h, tail.norm2, eps, residual=residual, residual_out=residual)
    logits = q8.gemm_mxfp4(tail.head, tail.head_scales, y)
    return q8.logprobs(logits, tokens, top=top)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--m", type=int, default=5)
    ap.add_argument("--k", type=int, default=4096)
    ap.add_argument("--vocab", type=int, default=64448)
    ap.add_argument("--top", type=int, default=5)
    ap.add_argument("--seed", type=int, default=0)
    a = ap.parse_args(argv)

    import torch
    from q8_block_quantized_act_gb300 import build as q8build

    q8build.build()
    g = torch.Generator(device="cuda").manual_seed(a.seed)

    def rnd(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    tail = make_tail(1 + 0.1 * rnd(a.k), 0.02 * rnd(a.k, a.k), 1 + 0.1 * rnd(a.k), 0.05 * rnd(a.vocab, a.k))
    tokens = torch.randint(0, a.vocab, (a.m,), generator=g, device="cuda").to(torch.int32)
    lp, entropy, ids, tlp = score(tail, rnd(a.m, a.k), rnd(a.m, a.k), tokens, top=a.top)
    torch.cuda.synchronize()
    q8.device_status()
    for t in range(min(a.m, 8)):
        best = ", ".join(f"{i} ({p:.3f})" for i, p in zip(ids[t].tolist(), tlp[t].tolist()))
        print(f"token {int(tokens[t])}: log p {float(lp[t]):.4f}, entropy {float(entropy[t]):.4f}, top {best}")
    print(f"{a.m} tokens, mean log p {float(lp.mean()):.4f}")


if __name__ == "__main__":
    main()
