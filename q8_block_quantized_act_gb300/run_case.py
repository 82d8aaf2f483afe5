"""Launch one kernel of libq8act on one shape, for profilers (no timing, no checking).

    python -m q8_block_quantized_act_gb300.run_case gemv --m 1 --n 64448 --k 4096 --reps 3
    python -m q8_block_quantized_act_gb300.run_case gemm --m 512 --n 4096 --k 4096 --reps 2

Kernels: quantize (q8_1), quantize_mmq, quantize_q8_0, gemv, gemm (fused quantize),
gemm_preq, gemm_repacked (fused quantize, load-time repacked weights), repack, dequant,
gemv_q4_0, dequant_q4_0, and the K-quant passes gemv_q6_k / gemv_q4_k / gemv_q5_k and
dequant_q6_k / dequant_q4_k / dequant_q5_k (on seeded random superblocks), norm and norm_mmq
(residual and weight, f16), quantize_mxfp4 and dequant_mxfp4 (f16), gemm_mxfp4 (f16 activation
quantized in the call, f16 out), logprobs (m rows of n f16 logits, 8 alternatives), and append_kv and
attention (m new tokens of one sequence of n positions, k / 128 query heads, k / 512 of keys, bf16, pages of 128).
Inputs are the seeded synthetic ones of q8_block_quantized_act_gb300.inputs;
one warm-up launch precedes the `--reps` launches.
"""
from __future__ import annotations

import argparse


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("kernel", choices=("quantize", "quantize_mmq", "quantize_q8_0", "gemv", "gemm",
                                       "gemm_preq", "gemm_repacked", "repack", "dequant", "gemv_q4_0",
                                       "dequant_q4_0", "gemv_q6_k", "gemv_q4_k", "gemv_q5_k",
                                       "dequant_q6_k", "dequant_q4_k", "dequant_q5_k", "norm", "norm_mmq",
                                       "quantize_mxfp4", "dequant_mxfp4", "gemm_mxfp4", "logprobs", "append_kv", "attention"))
    ap.add_argument("--m", type=int, default=1)
    ap.add_argument("--n", type=int, default=4096)
    ap.add_argument("--k", type=int, default=4096)
    ap.add_argument("--reps", type=int, default=1)
    a = ap.parse_args(argv)

    import torch
    import q8_block_quantized_act_gb300 as q8
    from q8_block_quantized_act_gb300 import build as q8build
    from q8_block_quantized_act_gb300 import inputs

    q8build.build()
    dev = torch.device("cuda")
    m, n, k = a.m, a.n, a.k
    x = torch.from_numpy(inputs.activations_f32(m, k)).to(dev)
    need_w = a.kernel in ("gemv", "gemm", "gemm_preq", "gemm_repacked", "repack", "dequant")
    w = q8.quantize_q8_0(torch.from_numpy(inputs.weights_f32(n, k)).to(dev)) if need_w else None
    w32 = torch.from_numpy(inputs.weights_f32(n, k)).to(dev) if a.kernel == "quantize_q8_0" else None
    w4 = (q8.quantize_q4_0(torch.from_numpy(inputs.weights_f32(n, k)).to(dev))
          if a.kernel in ("gemv_q4_0", "dequant_q4_0") else None)
    xq, xd = q8.quantize_q8_1(x)
    xqh, xdt = q8.quantize_q8_1_mmq(x)
    kq = a.kernel.split("_", 1)[1] if a.kernel.endswith("_k") else None   # "q6_k", "q4_k", "q5_k"
    wk = torch.from_numpy(inputs.kquant_superblocks(kq, n, k)).to(dev) if kq else None
    ws = q8.gemm_workspace(m, k, dev) if a.kernel in ("gemm", "gemm_repacked") else None
    wq16, wdt = q8.repack_q8_0(w, n, k) if a.kernel in ("gemm_repacked", "repack") else (None, None)
    x16 = x.half()
    if a.kernel in ("norm", "norm_mmq"):
        r16, g16 = x16.flip(0).contiguous(), torch.ones(k, dtype=torch.float16, device=dev)
    if a.kernel == "dequant_mxfp4":
        mx, out16 = q8.quantize_mxfp4(x16), torch.empty_like(x16)
    if a.kernel == "gemm_mxfp4":
        mx = q8.quantize_mxfp4(torch.from_numpy(inputs.weights_f32(n, k)).to(dev))
        mws, y16 = q8.gemm_mxfp4_workspace(m, k, dev), torch.empty((m, n), dtype=torch.float16, device=dev)
    if a.kernel == "logprobs":
        logits = torch.randn((m, n), device=dev).mul_(2.5).half()
        tok = torch.zeros(m, dtype=torch.int32, device=dev)
    if a.kernel in ("append_kv", "attention"):
        hq, hk, pages, i32 = k // 128, max(1, k // 512), -(-n // 128), dict(dtype=torch.int32, device=dev)
        kc, vc = (torch.randn((pages, hk, 128, 128), device=dev, dtype=torch.bfloat16) for _ in range(2))
        kv = q8.PagedKV(kc, vc, torch.arange(pages, **i32).view(1, -1), torch.tensor([0, m], **i32), torch.tensor([n], **i32))
        qkv = torch.randn((m, hq + 2 * hk, 128), device=dev, dtype=torch.bfloat16)
        parts = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        turns, aws, q16 = q8.rope_turns([10000.0 ** (-i / 64) for i in range(64)], dev), q8.attention_workspace(kv, hq), parts[0].contiguous()
    torch.cuda.synchronize()

    def once():
        if a.kernel == "append_kv":
            q8.append_kv(kv, *parts, turns=turns, out=q16)
        elif a.kernel == "attention":
            q8.attention(kv, q16, max_new=m, ws=aws)
        elif a.kernel == "norm":
            q8.rmsnorm_q8_1(x16, g16, residual=r16, residual_out=r16)
        elif a.kernel == "norm_mmq":
            q8.rmsnorm_q8_1_mmq(x16, g16, residual=r16, residual_out=r16)
        elif a.kernel == "quantize_mxfp4":
            q8.quantize_mxfp4(x16)
        elif a.kernel == "dequant_mxfp4":
            q8.dequant_mxfp4(*mx, out=out16)
        elif a.kernel == "gemm_mxfp4":
            q8.gemm_mxfp4(*mx, x16, ws=mws, out=y16)
        elif a.kernel == "logprobs":
            q8.logprobs(logits, tok, top=8)
        elif a.kernel == "quantize":
            q8.quantize_q8_1(x)
        elif a.kernel == "quantize_mmq":
            q8.quantize_q8_1_mmq(x)
        elif a.kernel == "quantize_q8_0":
            q8.quantize_q8_0(w32)
        elif a.kernel == "gemv":
            q8.gemv_q8_0(w, xq, xd, n)
        elif a.kernel == "gemm":
            q8.gemm_q8_0(w, x, n, ws=ws)
        elif a.kernel == "gemm_preq":
            q8.gemm_q8_0_preq(w, xqh, xdt, n)
        elif a.kernel == "gemm_repacked":
            q8.gemm_q8_0_repacked(wq16, wdt, x, ws=ws)
        elif a.kernel == "repack":
            q8.check(q8.q8act_repack_q8_0(w, wq16, wdt, n, k))
        elif a.kernel == "gemv_q4_0":
            q8.gemv_q4_0(w4, xq, xd, n)
        elif a.kernel == "dequant_q4_0":
            q8.dequant_q4_0_f16(w4, n, k)
        elif kq and a.kernel.startswith("gemv"):
            q8.gemv_kq(kq, wk, xq, xd, n)
        elif kq:
            q8.dequant_kq_f16(kq, wk, n, k)
        else:
            q8.dequant_q8_0_f16(w, n, k)

    for _ in range(1 + a.reps):
        once()
    torch.cuda.synchronize()
    q8.device_status()
    print(f"ran {a.kernel} m={m} n={n} k={k} x{1 + a.reps}")


if __name__ == "__main__":
    main()
