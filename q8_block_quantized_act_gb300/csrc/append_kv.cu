// append_kv.cu -- the new tokens' keys and values into the pages of the cache, their keys and
// queries rotated by their positions on the way.
//   turn = p * f_i mod 1 (f_i in turns a position),  (a, b) -> (a cos - b sin, b cos + a sin)
//
// Angles: f_i comes as a 64-bit fraction of a turn, so p * f_i mod 2^64 is the angle modulo one turn
// without any rounding however far the position; its upper 32 bits are rounded to f32 as half turns
// (2^-24 of the angle) and go through sincospif.
//
// A thread owns 16 values of a head: two vectors of 8 that are rotated against each other (halves), or
// 16 consecutive ones.  A CTA takes a few tokens, so that a token's sines and cosines are computed once
// and serve its heads; few tokens are spread over several CTAs by heads.
#include "launch.h"
#include "paged.cuh"
#include "types.cuh"

namespace q8 {
namespace {

constexpr int THREADS = 256;

struct Args {
    Paged p;
    const void *q, *k, *v;
    int64_t ldq, ldk, ldv, ldqo;
    void *kc, *vc, *qo;
    const uint64_t *turns;
    int hq, rot, interleaved;
};

struct Token {
    int64_t offset;      // of its slot's first head in the cache, or -1: it has no place there
    int row;             // or -1: behind the last sequence
};

// 16 values of T as f32, in two groups of 8.
template <typename T>
__device__ __forceinline__ void load16(const T *a, const T *b, float (&x)[16])
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint4 *p = reinterpret_cast<const uint4 *>(h ? b : a);
        if constexpr (sizeof(T) == 4) {
            float f[4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                unpack<T>(__ldg(p + i), f);
#pragma unroll
                for (int j = 0; j < 4; ++j) x[8 * h + 4 * i + j] = f[j];
            }
        } else {
            float f[8];
            unpack<T>(__ldg(p), f);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[8 * h + j] = f[j];
        }
    }
}

template <typename C>
__device__ __forceinline__ void store16(C *a, C *b, const float (&x)[16])
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = x[8 * h + j];
        *reinterpret_cast<uint4 *>(h ? b : a) = pack<C>(f);
    }
}

// T: the projection's type, C: the cache's, D: values a head, TOK: tokens a CTA.
template <typename T, typename C, int D, int TOK>
__global__ void __launch_bounds__(THREADS) append_kernel(Args a)
{
    __shared__ Token tok[TOK];
    __shared__ int s_pos[TOK];
    __shared__ alignas(16) float2 rotation[TOK][D / 2];      // (cos, sin)
    constexpr int UNITS = D / 16;                // of a head
    griddep_enter();
    const Paged &p = a.p;
    const int first = blockIdx.x * TOK;
    if (threadIdx.x < TOK) {
        const int row = first + threadIdx.x;
        Token t{-1, -1};
        int pos = 0;
        if (row < p.m) {
            int lo = 0, hi = p.seqs;             // the last sequence that starts at or before the row
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (__ldg(p.starts + mid) <= row) lo = mid;
                else hi = mid;
            }
            const Seq s = seq_of(p, lo);
            if (row >= s.row0 && row < s.row0 + s.n) {
                t.row = row;
                pos = s.pos0 + row - s.row0;
                if (pos >= 0 && pos < s.end) {
                    const int64_t page = page_of(p, lo, pos >> p.page_shift);
                    if (page >= 0) t.offset = page * p.page_stride + (int64_t)(pos & ((1 << p.page_shift) - 1)) * D;
                }
            }
        }
        tok[threadIdx.x] = t;
        s_pos[threadIdx.x] = pos;
    }
    __syncthreads();
    const int half = a.rot >> 1;
    for (int i = threadIdx.x; i < TOK * half; i += THREADS) {
        const int t = i / half, f = i - t * half;
        const uint64_t turn = (uint64_t)(int64_t)s_pos[t] * __ldg(a.turns + f);
        float sn, cs;
        sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &sn, &cs);
        rotation[t][f] = make_float2(cs, sn);
    }
    __syncthreads();

    const int hk = p.heads, heads = a.hq + 2 * hk, units = heads * UNITS;
    const int64_t head_stride = (int64_t)D << p.page_shift;
    // This CTA's part of the heads.
    const int u0 = (int)((int64_t)units * blockIdx.y / gridDim.y), u1 = (int)((int64_t)units * (blockIdx.y + 1) / gridDim.y);
    const int per = u1 - u0;
#pragma unroll 2
    for (int i = threadIdx.x; i < per * TOK; i += THREADS) {
        const int t = i / per, unit = u0 + i - t * per;
        const Token tk = tok[t];
        if (tk.row < 0) continue;
        const int head = unit / UNITS, u = unit % UNITS;
        const bool is_q = head < a.hq, is_v = head >= a.hq + hk;
        const int h = is_q ? head : is_v ? head - a.hq - hk : head - a.hq;
        const T *src = is_q   ? static_cast<const T *>(a.q) + tk.row * a.ldq
                       : is_v ? static_cast<const T *>(a.v) + tk.row * a.ldv
                              : static_cast<const T *>(a.k) + tk.row * a.ldk;
        const bool rotated = !is_v && 16 * u < a.rot;
        const bool halves = rotated && !a.interleaved;
        const int at0 = halves ? 8 * u : 16 * u, at1 = halves ? half + 8 * u : 16 * u + 8;
        src += h * D;
        C *dst;
        if (is_q) {
            dst = static_cast<C *>(a.qo) + tk.row * a.ldqo + h * D;
        } else {
            if (tk.offset < 0) continue;
            dst = static_cast<C *>(is_v ? a.vc : a.kc) + tk.offset + h * head_stride;
        }
        float x[16];
        load16(src + at0, src + at1, x);
        if (halves) {
            const float4 *r = reinterpret_cast<const float4 *>(&rotation[t][8 * u]);
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                const float4 cs = r[j / 2];
                const float a0 = x[j], b0 = x[8 + j], a1 = x[j + 1], b1 = x[9 + j];
                x[j] = a0 * cs.x - b0 * cs.y;
                x[8 + j] = b0 * cs.x + a0 * cs.y;
                x[j + 1] = a1 * cs.z - b1 * cs.w;
                x[9 + j] = b1 * cs.z + a1 * cs.w;
            }
        } else if (rotated) {
            const float4 *r = reinterpret_cast<const float4 *>(&rotation[t][8 * u]);
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                const float4 cs = r[j / 2];
                const float a0 = x[2 * j], b0 = x[2 * j + 1], a1 = x[2 * j + 2], b1 = x[2 * j + 3];
                x[2 * j] = a0 * cs.x - b0 * cs.y;
                x[2 * j + 1] = b0 * cs.x + a0 * cs.y;
                x[2 * j + 2] = a1 * cs.z - b1 * cs.w;
                x[2 * j + 3] = b1 * cs.z + a1 * cs.w;
            }
        }
        store16(dst + at0, dst + at1, x);
    }
}

}  // namespace

cudaError_t launch_append_kv(const DeviceInfo &dev, const q8act_paged_kv &kv, const AppendArgs &s, int64_t m,
                             cudaStream_t stream)
{
    const Args a{paged_of(kv, m), s.q, s.k, s.v, s.ldq, s.ldk, s.ldv, s.ldqo, kv.k, kv.v, s.q_out, s.turns, s.hq, s.rot,
                 s.interleaved};
    const int64_t units = (int64_t)(s.hq + 2 * kv.heads) * (kv.dim / 16);
    return with_type(s.type, [&](auto x) {
        return with_type(kv.type, [&](auto c) -> cudaError_t {
            using T = decltype(x);
            using C = decltype(c);
            if constexpr (sizeof(C) == 4) {
                return cudaErrorInvalidValue;
            } else {
                auto go = [&](auto kern, int tokens) {
                    const int64_t blocks = (m + tokens - 1) / tokens;
                    int64_t parts = dev.num_sms / blocks;
                    const int64_t most = (units * tokens + THREADS - 1) / THREADS;
                    parts = parts < 1 ? 1 : parts > most ? most : parts;
                    return launch_dependent(kern, dim3((unsigned)blocks, (unsigned)parts), THREADS, 0, stream, a);
                };
                if (m >= 4 * 4 * (int64_t)dev.num_sms)
                    return kv.dim == 64 ? go(append_kernel<T, C, 64, 4>, 4) : go(append_kernel<T, C, 128, 4>, 4);
                return kv.dim == 64 ? go(append_kernel<T, C, 64, 1>, 1) : go(append_kernel<T, C, 128, 1>, 1);
            }
        });
    });
}

}  // namespace q8
