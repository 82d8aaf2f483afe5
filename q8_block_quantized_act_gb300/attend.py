"""The attention block of a decoder layer: block-quantized projections around a paged cache.

    python -m q8_block_quantized_act_gb300.attend --prompt 700 --steps 4

For m new tokens' hidden states x and their residual stream:

    residual += x; norm; q8_1           rmsnorm_q8_1 (m <= 15) or rmsnorm_q8_1_mmq
    q, k, v = projection (Q8_0 x q8_1)  gemv_q8_0 (m <= 15) or gemm_q8_0_preq
    rotation; k, v into the cache       append_kv
    attention over the cache            attention
    h = output projection (Q8_0)        gemv_q8_0 (m <= 15) or gemm_q8_0

on one stream, no host synchronization between the calls; a captured step is replayed as the sequences
grow.  The command takes a synthetic prompt through the block in two chunks, decodes a few tokens with a
captured graph and prints how far the decoded outputs are from those of the whole in one chunk.
"""
from __future__ import annotations

import argparse
from dataclasses import dataclass

import q8_block_quantized_act_gb300 as q8
from q8_block_quantized_act_gb300.score_tokens import project


@dataclass
class Block:
    """Weights: a norm, Q8_0 projections [(heads_q + 2 heads) dim, k] and [k, heads_q dim], rotation."""
    norm: object
    qkv: object           # Q8_0 bytes
    out: object           # Q8_0 bytes
    turns: object
    heads_q: int
    heads: int
    dim: int


def make_block(norm, qkv, out, heads_q: int, heads: int, dim: int, base: float = 10000.0) -> Block:
    """Quantize float32 CUDA weights once, at load time."""
    turns = q8.rope_turns([base ** (-2 * i / dim) for i in range(dim // 2)], norm.device)
    return Block(norm, q8.quantize_q8_0(qkv), q8.quantize_q8_0(out), turns, heads_q, heads, dim)


def attend(block: Block, kv, x, residual, max_new=None, ws=None, eps: float = 1e-6):
    """x, residual [m, k] float32 (the residual stream is updated in place), kv a PagedKV of the m new
    tokens, max_new as attention takes it (1 when decoding) -> the block's output [m, k] float32."""
    m, k = x.shape
    hq, hk, d = block.heads_q, block.heads, block.dim
    n = (hq + 2 * hk) * d
    few = m <= q8.Q8ACT_GEMV_MAX_M
    if few:
        xq, xd = q8.rmsnorm_q8_1(x, block.norm, eps, residual=residual, residual_out=residual)
        y = project(block.qkv, xq, xd, n, x.new_empty((m, n)))
    else:
        xqh, xdt = q8.rmsnorm_q8_1_mmq(x, block.norm, eps, residual=residual, residual_out=residual)
        y = q8.gemm_q8_0_preq(block.qkv, xqh, xdt, n)
    y = y.view(m, hq + 2 * hk, d)
    q = q8.append_kv(kv, y[:, :hq], y[:, hq:hq + hk], y[:, hq + hk:], turns=block.turns)
    o = q8.attention(kv, q, max_new=max_new, ws=ws, dtype=x.dtype).view(m, hq * d)
    if few:
        oq, od = q8.quantize_q8_1(o)
        return project(block.out, oq, od, k, x.new_empty((m, k)))
    return q8.gemm_q8_0(block.out, o, k)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--prompt", type=int, default=700)
    ap.add_argument("--steps", type=int, default=4)
    ap.add_argument("--k", type=int, default=4096)
    ap.add_argument("--seed", type=int, default=0)
    a = ap.parse_args(argv)

    import torch
    from q8_block_quantized_act_gb300 import build as q8build

    q8build.build()
    g = torch.Generator(device="cuda").manual_seed(a.seed)

    def rnd(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    hq, hk, d, page = a.k // 128, max(1, a.k // 512), 128, 64
    block = make_block(1 + 0.1 * rnd(a.k), 0.02 * rnd((hq + 2 * hk) * d, a.k), 0.02 * rnd(a.k, hq * d), hq, hk, d)
    total = a.prompt + a.steps
    pages = -(-total // page)
    x = rnd(total, a.k)

    def batch(length, new):
        k, v = (torch.zeros((pages, hk, page, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        i32 = dict(dtype=torch.int32, device="cuda")
        table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).view(1, -1)
        return q8.PagedKV(k, v, table, torch.tensor([0, new], **i32), torch.tensor([length], **i32))

    whole = attend(block, batch(total, total), x, torch.zeros_like(x))

    kv = batch(0, 0)
    outs, at = [], 0
    for new in (a.prompt // 2, a.prompt - a.prompt // 2):
        if new:
            kv.lens += new
            kv.starts[1] = new
            part = x[at:at + new]
            outs.append(attend(block, kv, part, torch.zeros_like(part)))
            at += new
    one, ws = x[:1].clone(), q8.attention_workspace(kv, hq)
    residual = torch.zeros_like(one)
    kv.starts[1] = 1
    kv.lens += 1
    step = lambda: attend(block, kv, one, residual, max_new=1, ws=ws)     # noqa: E731
    step()                                            # once outside: loads what a capture may not
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h = step()
    kv.lens -= 1
    for i in range(a.steps):
        one.copy_(x[at + i:at + i + 1])
        residual.zero_()
        kv.lens += 1
        graph.replay()
        outs.append(h.clone())
    torch.cuda.synchronize()
    q8.device_status()
    got = torch.cat(outs)
    for name, s in (("prompt in two chunks", slice(0, a.prompt)), ("decoded one by one", slice(a.prompt, total))):
        if got[s].numel():
            print(f"{name}: {got[s].shape[0]} tokens, off by {float((got[s] - whole[s]).norm() / whole[s].norm()):.2e} "
                  "of the whole in one chunk")


if __name__ == "__main__":
    main()
