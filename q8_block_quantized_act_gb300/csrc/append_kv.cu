// append_kv.cu -- the new tokens' keys and values into the pages of the cache, their keys and
// queries rotated by their positions on the way.
//   turn = p * f_i mod 1 (f_i in turns a position),  (a, b) -> (a cos - b sin, b cos + a sin)
//
// Angles: f_i comes as a 64-bit fraction of a turn, so p * f_i mod 2^64 is the angle modulo one turn
// without any rounding however far the position; its upper 32 bits are rounded to f32 as half turns
// (2^-24 of the angle) and go through sincospif.
//
// A thread owns 16 values of a head: two vectors of 8 that are rotated against each other (halves), or
// 16 consecutive ones.  A CTA takes one or two tokens, so that a token's sines and cosines are computed once
// and serve its heads; few tokens are spread over several CTAs by heads.  The first values' loads are issued
// before the chain starts -> length -> page -> angle, which no bytes pass during.
//
// Bound by memory: 8191 tokens of 32 + 8 heads x 128 bf16 36.5 us (5.5 TB/s, 0.81 of a copy; one token 3.4 us: launch
// and that chain).  What is missing is that chain, about 1 us of each CTA's 5: more values ahead in registers leave
// fewer CTAs to an SM and lost (256 threads x 4 tokens ahead 46.7 us, x 2 40.7).
#include "launch.h"
#include "paged.cuh"
#include "types.cuh"

namespace q8 {
namespace {

constexpr int THREADS = 128;

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

// 16 values of T, two groups of 8, on their way.
template <typename T>
struct Sixteen {
    uint4 w[sizeof(T)];
    __device__ __forceinline__ void load(const T *a, const T *b)
    {
        constexpr int N = sizeof(T) / 2;             // vectors of 8 values
#pragma unroll
        for (int i = 0; i < N; ++i) {
            w[i] = __ldcs(reinterpret_cast<const uint4 *>(a) + i);
            w[N + i] = __ldcs(reinterpret_cast<const uint4 *>(b) + i);
        }
    }
    __device__ __forceinline__ void values(float (&x)[16]) const
    {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T); ++i) {
            float f[VEC<T>];
            unpack<T>(w[i], f);
#pragma unroll
            for (int j = 0; j < VEC<T>; ++j) x[VEC<T> * i + j] = f[j];
        }
    }
};

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

// A thread's 16 values of a token: where they are read and, of each token, written.
template <typename T, typename C, int D>
struct Place {
    const T *src;            // of token row 0
    C *dst;                  // of row 0, or of the cache's first slot
    int64_t ld;
    int at0, at1, u;
    bool is_q, halves, rotated;

    __device__ __forceinline__ Place(const Args &a, int unit)
    {
        constexpr int UNITS = D / 16;
        const int hk = a.p.heads, head = unit / UNITS;
        u = unit % UNITS;
        is_q = head < a.hq;
        const bool is_v = head >= a.hq + hk;
        const int h = is_q ? head : is_v ? head - a.hq - hk : head - a.hq;
        ld = is_q ? a.ldq : is_v ? a.ldv : a.ldk;
        rotated = !is_v && 16 * u < a.rot;
        halves = rotated && !a.interleaved;
        at0 = halves ? 8 * u : 16 * u;
        at1 = halves ? (a.rot >> 1) + 8 * u : 16 * u + 8;
        src = static_cast<const T *>(is_q ? a.q : is_v ? a.v : a.k) + h * D;
        dst = is_q ? static_cast<C *>(a.qo) + h * D
                   : static_cast<C *>(is_v ? a.vc : a.kc) + h * ((int64_t)D << a.p.page_shift);
    }
};

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
    // This CTA's part of the heads.  The first values are under way while positions, pages and angles are worked out.
    const int units = (a.hq + 2 * p.heads) * UNITS;
    const int u0 = (int)((int64_t)units * blockIdx.y / gridDim.y), u1 = (int)((int64_t)units * (blockIdx.y + 1) / gridDim.y);
    int unit = u0 + threadIdx.x;
    Sixteen<T> w[TOK];
    auto load = [&](const Place<T, C, D> &at) {
#pragma unroll
        for (int t = 0; t < TOK; ++t)
            if (first + t < p.m) w[t].load(at.src + (first + t) * at.ld + at.at0, at.src + (first + t) * at.ld + at.at1);
    };
    if (unit < u1) load(Place<T, C, D>(a, unit));
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

    for (; unit < u1; unit += THREADS) {
        const Place<T, C, D> at(a, unit);
        if (unit >= u0 + THREADS) load(at);
#pragma unroll
        for (int t = 0; t < TOK; ++t) {
            const Token tk = tok[t];
            if (tk.row < 0 || (!at.is_q && tk.offset < 0)) continue;
            C *dst = at.dst + (at.is_q ? tk.row * a.ldqo : tk.offset);
            float x[16];
            w[t].values(x);
            const float4 *r = reinterpret_cast<const float4 *>(&rotation[t][8 * at.u]);
            if (at.halves) {
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    const float4 cs = r[j / 2];
                    const float a0 = x[j], b0 = x[8 + j], a1 = x[j + 1], b1 = x[9 + j];
                    x[j] = a0 * cs.x - b0 * cs.y;
                    x[8 + j] = b0 * cs.x + a0 * cs.y;
                    x[j + 1] = a1 * cs.z - b1 * cs.w;
                    x[9 + j] = b1 * cs.z + a1 * cs.w;
                }
            } else if (at.rotated) {
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
            store16(dst + at.at0, dst + at.at1, x);
        }
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
                // Two tokens a CTA share its sines' latency: 8191 tokens of 32 + 8 heads x 128 bf16 36.5 us, one by one
                // 37.8, four 39.6; 64 values 18.4 and 20.8; 1000 tokens of 128 values 7.4 and 8.3.  From f32 rows two need 74
                // registers, one 58, and lose: 8191 tokens 49.4 (0.90 of a copy) and 48.3, 1000 tokens 10.8 and 8.5, 64 values
                // the same 24.5.  Few tokens are worth a CTA each (62 tokens: the same 3.8 us).
                if (m >= 4 * (int64_t)dev.num_sms)
                    return kv.dim == 64 ? go(append_kernel<T, C, 64, 2>, 2) : go(append_kernel<T, C, 128, 2>, 2);
                return kv.dim == 64 ? go(append_kernel<T, C, 64, 1>, 1) : go(append_kernel<T, C, 128, 1>, 1);
            }
        });
    });
}

}  // namespace q8
