// attention.cu -- causal attention of a few new tokens a sequence (one: decoding) over a paged cache.
//   s_j = scale q . k_j,  o = sum_j e^(s_j - mx) v_j / sum_j e^(s_j - mx)  over the visible positions j
//
// Bound by memory: each key and value is read once and serves the group's query heads.  A CTA walks
// over the units of the batch (attention.cuh), so that 152 SMs are filled whatever the number and the
// lengths of the sequences.  One warp brings 64 positions at a time to shared memory (TMA boxes of up to
// a page, 128-byte swizzled, several stages ahead across units); four warps take 16 positions each,
// with their own running maximum and sum, so they meet only at the end of a unit.  The products run on
// the warp-level tensor-core MMA: 16 rows are too few for tcgen05's 128, and it is not what bounds.
// Scores, statistics and sums are f32; the weights e^(s - mx) <= 1 are rounded to the cache's type for
// the second product, whose operands have one type.
#include <algorithm>

#include "attention.cuh"

namespace q8 {
namespace {

constexpr int TILE = 64;             // positions a stage
constexpr int CONSUMERS = 4;         // warps, 16 positions each
constexpr int THREADS = 32 * (CONSUMERS + 1);
constexpr int ROWS = 16;
constexpr int COUNTERS = 128;        // threads that count the units
constexpr float NEG = -INFINITY;

template <int D>
struct Cfg {
    static constexpr int TILE_BYTES = TILE * D * 2;             // of keys, and of values
    static constexpr int STAGE_BYTES = 2 * TILE_BYTES;
    static constexpr int STAGES = 96 * 1024 / STAGE_BYTES;      // two CTAs to an SM
    static constexpr int HALVES = D / 64;                       // 128-byte wide columns of a tile
};

struct Shared {
    PlanSmem<COUNTERS> plan;
    uint64_t full[8], empty[8];
    uint32_t ok[8];                       // a stage's 16-position blocks whose page exists
    float mx[2][CONSUMERS][ROWS], sum[2][CONSUMERS][ROWS];
    int spoilt[2][CONSUMERS];             // a non-finite value that not all rows see
    int abort_flag;
};

template <typename T>
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if constexpr (std::is_same<T, __half>::value) {
        mma_f16_16816(d, a, b0, b1, d);
    } else {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t saddr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(saddr) : "memory");
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t saddr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(saddr) : "memory");
}

// Two f32 rounded to the low and the high half of a word.
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    if constexpr (std::is_same<T, __half>::value) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

// Whether a word's low or high half is an infinity or NaN.
template <typename T>
__device__ __forceinline__ bool non_finite2(uint32_t w)
{
    constexpr uint32_t E = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
    return (w & E) == E || (w >> 16 & E) == E;
}

template <typename T, int D>
__global__ void __launch_bounds__(THREADS, 2)
    attention_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, Attn a)
{
    using C = Cfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *stages = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    Shared &sm = *reinterpret_cast<Shared *>(stages + C::STAGES * C::STAGE_BYTES);
    volatile int *abort_flag = &sm.abort_flag;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) { mbar_init(&sm.full[s], 1); mbar_init(&sm.empty[s], CONSUMERS); }
        sm.abort_flag = 0;
        fence_mbar_init();
    }
    griddep_wait();
    griddep_launch_dependents();
    Plan<ROWS, TILE, COUNTERS> plan;
    plan.make(a, sm.plan);                                       // and the barriers exist for all

    if (warp == CONSUMERS) {
        // ------------------------------ producer ------------------------------
        const int ps = 1 << a.p.page_shift, per_tile = ps < TILE ? TILE / ps : 1, blocks = 4 / per_tile;
        int it = 0, st = 0;
        uint32_t phase = 1;
        bool ok = true;
        for (int u = blockIdx.x; ok && u < plan.total; u += gridDim.x) {
            const Unit x = plan.find(a, sm.plan, u);
            const int rows = x.s.n * a.group, r0 = x.tile * ROWS, r1 = min(r0 + ROWS, rows) - 1;
            const Span span = span_of<TILE>(a, x.s, r0, r1);
            int t0, t1;
            span.part(x.part, x.parts, t0, t1);
            for (int t = t0; t < t1; ++t, ++it) {
                const int pos = t * TILE;
                const int64_t page = lane < per_tile ? page_of(a.p, x.b, (pos >> a.p.page_shift) + lane) : -1;
                const uint32_t good = __ballot_sync(0xffffffffu, page >= 0);
                uint32_t okm = 0;
                for (int j = 0; j < per_tile; ++j)
                    if (good >> j & 1) okm |= ((1u << blocks) - 1) << (j * blocks);
                // A page that does not exist: a box outside the tensor, which reads as zeros.
                const int id = page < 0 ? (int)a.p.pages : (int)page;
                ok = __all_sync(0xffffffffu, wait_or_abort(&sm.empty[st], phase, a.status, abort_flag));
                if (!ok) break;
                if (lane == 0) {
                    sm.ok[st] = okm;
                    mbar_arrive_expect_tx(&sm.full[st], C::STAGE_BYTES);
                }
                __syncwarp();
                for (int i0 = 0; i0 < 2 * C::HALVES * per_tile; i0 += 32) {
                    const int i = i0 + lane, j = i / (2 * C::HALVES), half = i % C::HALVES, is_v = i / C::HALVES % 2;
                    const int box_page = __shfl_sync(0xffffffffu, id, j & 31);
                    if (i < 2 * C::HALVES * per_tile)
                        tma_load_4d(stages + st * C::STAGE_BYTES + is_v * C::TILE_BYTES + half * (TILE * 128) + j * ps * 128,
                                    is_v ? &tm_v : &tm_k, half * 64, ps > TILE ? pos & (ps - 1) : 0, x.h, box_page,
                                    &sm.full[st]);
                }
                if (++st == C::STAGES) {
                    st = 0;
                    phase ^= 1;
                }
            }
        }
        // Never leave with a copy into this CTA's shared memory in flight.
        for (int i = it > C::STAGES ? it - C::STAGES : 0; i < it; ++i)
            mbar_wait_drain(&sm.full[i % C::STAGES], (i / C::STAGES) & 1, a.status);
        return;
    }

    // ------------------------------ consumers ------------------------------
    const int g = lane >> 2, c = lane & 3;
    const uint32_t stage0 = smem_u32(stages);
    // Rows of this lane's ldmatrix addresses: keys in their own order, values transposed.
    const int krow = warp * 16 + (lane & 7) + (lane >> 4) * 8, kchunk = lane >> 3 & 1;
    const int vrow = warp * 16 + (lane & 7) + (lane >> 3 & 1) * 8, vchunk = lane >> 4;
    int it = 0, st = 0, flip = 0;
    uint32_t phase = 0;
    for (int u = blockIdx.x; u < plan.total; u += gridDim.x) {
        const Unit x = plan.find(a, sm.plan, u);
        const int rows = x.s.n * a.group, r0 = x.tile * ROWS, valid = min(ROWS, rows - r0);
        const Span span = span_of<TILE>(a, x.s, r0, r0 + valid - 1);
        int t0, t1;
        span.part(x.part, x.parts, t0, t1);
        const int first = x.s.pos0 + a.by_group(r0), last = x.s.pos0 + a.by_group(r0 + valid - 1);    // positions of its rows

        // Two rows a lane: g and g + 8.
        uint32_t q[D / 16][4];
        int lo[2], hi[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = r0 + g + 8 * i;
            const bool live = r < rows;
            const int tok = live ? a.by_group(r) : 0;
            const int pos = x.s.pos0 + tok;
            hi[i] = live ? min(pos, x.s.end - 1) : -1;
            lo[i] = a.window ? max(pos - a.window + 1, 0) : 0;
            const uint32_t *src = reinterpret_cast<const uint32_t *>(
                static_cast<const T *>(a.q) + (x.s.row0 + tok) * a.ldq + (x.h * a.group + (live ? r - tok * a.group : 0)) * D) + c;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                q[kk][i] = live ? __ldg(src + kk * 8) : 0u;
                q[kk][i + 2] = live ? __ldg(src + kk * 8 + 4) : 0u;
            }
        }
        float o[D / 8][4], mx[2] = {NEG, NEG}, sum[2] = {0.0f, 0.0f};
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[n][i] = 0.0f;
        bool aborted = false, spoilt = false;

        for (int t = t0; t < t1; ++t, ++it) {
            aborted = !__all_sync(0xffffffffu, wait_or_abort(&sm.full[st], phase, a.status, abort_flag));
            if (aborted) break;
            const uint32_t kt = stage0 + st * C::STAGE_BYTES, vt = kt + C::TILE_BYTES;
            const bool page_ok = sm.ok[st] >> warp & 1;
            float s[2][4] = {};
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                uint32_t kf[4];
                const int chunk = kk * 2 + kchunk;
                ldmatrix_x4(kf, kt + (chunk >> 3) * (TILE * 128) + krow * 128 + (((chunk & 7) ^ (krow & 7)) << 4));
                mma_16816<T>(s[0], q[kk], kf[0], kf[1]);
                mma_16816<T>(s[1], q[kk], kf[2], kf[3]);
            }
            // Columns of s[n]: positions key0 + 8 n + 2 c and the next; rows g (0, 1) and g + 8 (2, 3).
            const int key0 = t * TILE + warp * 16;
            // Whether some row does not see some of the 16.
            const bool part = key0 < span.lo || key0 + 15 > min(first, span.hi) || (a.window && key0 <= last - a.window) || !page_ok;
            if (part) {
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int key = key0 + 8 * n + 2 * c + (i & 1);
                        if (key < lo[i >> 1] || key > hi[i >> 1] || !page_ok) s[n][i] = NEG;
                    }
            }
            uint32_t p[4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float m = fmaxf(fmaxf(s[0][2 * i], s[0][2 * i + 1]), fmaxf(s[1][2 * i], s[1][2 * i + 1]));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
                m = fmaxf(mx[i], m * a.scale);
                if (__any_sync(0xffffffffu, m > mx[i])) {
                    const float f = attn_ex2(mx[i] - (m == NEG ? 0.0f : m));
                    sum[i] *= f;
#pragma unroll
                    for (int n = 0; n < D / 8; ++n) {
                        o[n][2 * i] *= f;
                        o[n][2 * i + 1] *= f;
                    }
                    mx[i] = m;
                }
                const float base = m == NEG ? 0.0f : m;
                float e[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) e[j] = attn_ex2(fmaf(s[j >> 1][2 * i + (j & 1)], a.scale, -base));
                sum[i] += (e[0] + e[1]) + (e[2] + e[3]);
                p[i] = pack2<T>(e[0], e[1]);
                p[i + 2] = pack2<T>(e[2], e[3]);
            }
            // Values of positions that no row sees are cleared.
            uint32_t keep[2] = {~0u, ~0u};
            if (part) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int key = key0 + 8 * i + 2 * c;
                    keep[i] = (key >= span.lo && key <= span.hi ? 0xffffu : 0u) |
                              (key + 1 >= span.lo && key + 1 <= span.hi ? 0xffff0000u : 0u);
                }
            }
#pragma unroll
            for (int n = 0; n < D / 16; ++n) {
                uint32_t vf[4];
                const int chunk = 2 * n + vchunk;
                ldmatrix_x4_trans(vf, vt + (chunk >> 3) * (TILE * 128) + vrow * 128 + (((chunk & 7) ^ (vrow & 7)) << 4));
                if (part) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        vf[i] &= keep[i & 1];
                        spoilt |= non_finite2<T>(vf[i]);
                    }
                }
                mma_16816<T>(o[2 * n], p, vf[0], vf[1]);
                mma_16816<T>(o[2 * n + 1], p, vf[2], vf[3]);
            }
            // The unit's last stage is handed back after the join, which uses its memory.
            if (t + 1 < t1) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.empty[st]);
                if (++st == C::STAGES) {
                    st = 0;
                    phase ^= 1;
                }
            }
        }

        // ---- join of the four warps ----
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
            sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
            if (c == 0) {
                sm.mx[flip][warp][g + 8 * i] = mx[i];
                sm.sum[flip][warp][g + 8 * i] = sum[i];
            }
        }
        spoilt = __any_sync(0xffffffffu, spoilt);
        if (lane == 0) sm.spoilt[flip][warp] = spoilt;
        if (bar_red_or(1, 32 * CONSUMERS, aborted)) return;
        const bool some = t1 > t0;
        float *join = reinterpret_cast<float *>(stages + st * C::STAGE_BYTES);      // [warp][row][D], 16-byte words swizzled by row
        if (some) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = g + 8 * i;
                float m = NEG;
#pragma unroll
                for (int w = 0; w < CONSUMERS; ++w) m = fmaxf(m, sm.mx[flip][w][r]);
                const float f = attn_ex2(mx[i] - (m == NEG ? 0.0f : m));
#pragma unroll
                for (int n = 0; n < D / 8; ++n) {
                    const int col = (8 * n + 2 * c) ^ ((r & 7) << 2);
                    *reinterpret_cast<float2 *>(join + (warp * ROWS + r) * D + col) = make_float2(o[n][2 * i] * f, o[n][2 * i + 1] * f);
                }
            }
            named_bar_sync(2, 32 * CONSUMERS);
        }
        {
            const int r = threadIdx.x >> 3, c8 = threadIdx.x & 7;        // a row, and every eighth vector of it
            if (r < valid) {
                float m = NEG, l = 0.0f;
#pragma unroll
                for (int w = 0; w < CONSUMERS; ++w) m = fmaxf(m, sm.mx[flip][w][r]);
                const float base = m == NEG ? 0.0f : m;
#pragma unroll
                for (int w = 0; w < CONSUMERS; ++w) l += sm.sum[flip][w][r] * attn_ex2(sm.mx[flip][w][r] - base);
                float acc[D / 8];
#pragma unroll
                for (int j = 0; j < D / 8; ++j) acc[j] = 0.0f;
                if (some) {
#pragma unroll
                    for (int w = 0; w < CONSUMERS; ++w)
#pragma unroll
                        for (int j = 0; j < D / 32; ++j) {
                            const float4 v = *reinterpret_cast<const float4 *>(
                                join + (w * ROWS + r) * D + (((j * 8 + c8) ^ (r & 7)) << 2));
                            acc[4 * j] += v.x;
                            acc[4 * j + 1] += v.y;
                            acc[4 * j + 2] += v.z;
                            acc[4 * j + 3] += v.w;
                        }
                }
                const int row = r0 + r, tok = a.by_group(row), head = x.h * a.group + row - tok * a.group;
                const int *sp = sm.spoilt[flip];
                if (sp[0] | sp[1] | sp[2] | sp[3]) {
                    const int pos = x.s.pos0 + tok;
                    const int k0 = max(a.window ? pos - a.window + 1 : 0, t0 * TILE), k1 = min(min(pos, x.s.end - 1), t1 * TILE - 1);
                    exact_values<T, D>(a, x.b, x.h, static_cast<const T *>(a.q) + (x.s.row0 + tok) * a.ldq + head * D, k0, k1,
                                       base, [&](int j) { return ((j >> 2) * 8 + c8) * 4 + (j & 3); }, acc);
                }
                if (x.parts > 1) {
                    const int64_t at = (int64_t)(x.slot + x.part) * ROWS + r;
                    if (c8 == 0) a.ml[at] = make_float2(m, l);
#pragma unroll
                    for (int j = 0; j < D / 32; ++j)
                        *reinterpret_cast<float4 *>(a.part + at * D + (j * 8 + c8) * 4) =
                            make_float4(acc[4 * j], acc[4 * j + 1], acc[4 * j + 2], acc[4 * j + 3]);
                } else {
                    const float inv = l == 0.0f ? 0.0f : 1.0f / l;       // a row that sees nothing: 0
                    uint8_t *dst = static_cast<uint8_t *>(a.out) +
                                   ((x.s.row0 + tok) * a.ldo + head * D) * out_size(a.otype);
#pragma unroll
                    for (int j = 0; j < D / 32; ++j)
                        store4(dst + (j * 8 + c8) * 4 * out_size(a.otype), a.otype,
                               make_float4(acc[4 * j] * inv, acc[4 * j + 1] * inv, acc[4 * j + 2] * inv, acc[4 * j + 3] * inv));
                }
            }
        }
        if (some) {
            fence_proxy_async_smem();            // the join's words before the next copies to the stage
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.empty[st]);
            if (++st == C::STAGES) {
                st = 0;
                phase ^= 1;
            }
        }
        // The next unit's statistics go to the other words: some warps may still read these.  They are
        // written again only behind the next unit's barrier.
        flip ^= 1;
    }
}

// ---------------------------------------------------------------------------------------
// Row tiles in several parts: o = sum_i e^(mx_i - mx) o_i / sum_i e^(mx_i - mx) sum_i, added in the parts' order.
// Few rows come in many parts (decoding), which W warps of a CTA share; many rows in few, a row a warp.
// ---------------------------------------------------------------------------------------
// The kernel works out which rows it joins while the parts are still being computed.
// ---------------------------------------------------------------------------------------
constexpr int JOIN_WARPS = 4;

template <int D, int ROWS_, int TILE_, int NT, int W>
__global__ void __launch_bounds__(32 * JOIN_WARPS) attention_join_kernel(Attn a)
{
    constexpr int V = D / 32;                // values a lane
    __shared__ PlanSmem<NT> sm;
    __shared__ alignas(16) float acc[W > 1 ? W : 1][D];
    __shared__ float mw[W], lw[W];
    const int warp = W > 1 ? threadIdx.x >> 5 : 0, lane = threadIdx.x & 31;
    // (what starts, lens and the table hold was there before the kernel in front, which has waited for it)
    Plan<ROWS_, TILE_, NT> plan;
    plan.make(a, sm);
    const int n = sm.items[NT];
    // A CTA's rows one by one, first rows first (the last of a row tile may not be there); or a warp's in fours.
    constexpr int R = W > 1 ? 1 : 4;
    const int work = n * (ROWS_ / R), step = gridDim.x * (JOIN_WARPS / W);
    bool waited = false;
    for (int i = blockIdx.x * (JOIN_WARPS / W) + (W > 1 ? 0 : threadIdx.x >> 5); i < work; i += step) {
        const int i0 = W > 1 ? i / n : i % (ROWS_ / R) * R;
        const Unit it = plan.find_item(a, sm, W > 1 ? i - i0 * n : i / (ROWS_ / R));
        if (!waited) griddep_enter();
        waited = true;
        const int rows = it.s.n * a.group - it.tile * ROWS_;
#pragma unroll 1
        for (int r = i0; r < min(i0 + R, rows); ++r) {
            const int row = it.tile * ROWS_ + r;
            const float2 *ml = a.ml + (int64_t)it.slot * ROWS_ + r;
            const float *part = a.part + ((int64_t)it.slot * ROWS_ + r) * D + V * lane;
            float m = NEG;
            for (int s = warp * 32 + lane; s < it.parts; s += 32 * W) m = fmaxf(m, ml[(int64_t)s * ROWS_].x);
#pragma unroll
            for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            if constexpr (W > 1) {
                if (lane == 0) mw[warp] = m;
                __syncthreads();
#pragma unroll
                for (int w = 0; w < W; ++w) m = fmaxf(m, mw[w]);
            }
            const float base = m == NEG ? 0.0f : m;
            float l = 0.0f, v[V] = {};
            const int s0 = it.parts * warp / W, s1 = it.parts * (warp + 1) / W;
#pragma unroll 4
            for (int s = s0; s < s1; ++s) {
                const float2 ms = ml[(int64_t)s * ROWS_];
                const float f = attn_ex2(ms.x - base);
                l = fmaf(ms.y, f, l);
                float w[V];
                if constexpr (V == 4) {
                    const float4 u = *reinterpret_cast<const float4 *>(part + (int64_t)s * ROWS_ * D);
                    w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
                } else {
                    const float2 u = *reinterpret_cast<const float2 *>(part + (int64_t)s * ROWS_ * D);
                    w[0] = u.x; w[1] = u.y;
                }
#pragma unroll
                for (int j = 0; j < V; ++j) v[j] = fmaf(w[j], f, v[j]);
            }
            const int tok = a.by_group(row), head = it.h * a.group + row - tok * a.group;
            uint8_t *dst = static_cast<uint8_t *>(a.out) + ((it.s.row0 + tok) * a.ldo + head * D) * out_size(a.otype);
            if constexpr (W > 1) {
#pragma unroll
                for (int j = 0; j < V; ++j) acc[warp][V * lane + j] = v[j];
                if (lane == 0) lw[warp] = l;
                __syncthreads();
                if (threadIdx.x < D / 4) {
                    float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    l = 0.0f;
#pragma unroll
                    for (int w = 0; w < W; ++w) {
                        const float4 u = *reinterpret_cast<const float4 *>(&acc[w][4 * threadIdx.x]);
                        t.x += u.x; t.y += u.y; t.z += u.z; t.w += u.w;
                        l += lw[w];
                    }
                    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                    store4(dst + 4 * threadIdx.x * out_size(a.otype), a.otype, make_float4(t.x * inv, t.y * inv, t.z * inv, t.w * inv));
                }
                __syncthreads();
            } else {
                const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                if constexpr (V == 4) {
                    store4(dst + 4 * lane * out_size(a.otype), a.otype, make_float4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv));
                } else {
                    const float x = __shfl_down_sync(0xffffffffu, v[0] * inv, 1), y = __shfl_down_sync(0xffffffffu, v[1] * inv, 1);
                    if (!(lane & 1)) store4(dst + 2 * lane * out_size(a.otype), a.otype, make_float4(v[0] * inv, v[1] * inv, x, y));
                }
            }
        }
    }
    if (!waited) griddep_enter();
}

}  // namespace

cudaError_t launch_attention_chunk_join(const DeviceInfo &dev, const Attn &a, int dim, cudaStream_t stream)
{
    auto go = [&](auto kern) { return launch_dependent(kern, dim3(4 * dev.num_sms), 32 * JOIN_WARPS, 0, stream, a); };
    return dim == 64 ? go(attention_join_kernel<64, CHUNK_ROWS, CHUNK_TILE, CHUNK_COUNTERS, 1>)
                     : go(attention_join_kernel<128, CHUNK_ROWS, CHUNK_TILE, CHUNK_COUNTERS, 1>);
}

// Partial results: of four rounds of a GB300's 152 SMs at two CTAs each, twice (Plan::make).
constexpr int SLOTS = 2 * 4 * 2 * 152;

size_t attention_workspace_bytes(int dim)
{
    return std::max(attention_space(SLOTS, ROWS, dim), attention_chunk_space(dim));
}

cudaError_t launch_attention(const DeviceInfo &dev, const q8act_paged_kv &kv, const AttentionArgs &s, int64_t m,
                             cudaStream_t stream)
{
    Attn a{};
    a.p = paged_of(kv, m);
    a.kc = kv.k;
    a.vc = kv.v;
    a.q = s.q;
    a.out = s.out;
    a.ldq = s.ldq;
    a.ldo = s.ldo;
    a.group = s.hq / kv.heads;
    a.by_group = Divide(a.group);
    a.by_heads = Divide(kv.heads);
    a.otype = s.otype;
    a.window = s.window;
    a.scale = s.scale * 1.4426950408889634f;
    a.status = dev.status;
    const int64_t most = s.max_new && s.max_new < m ? s.max_new : m;     // new tokens of a sequence
    if (most * a.group > ROWS) return launch_attention_chunk(dev, kv, a, s.ws, stream);
    attention_place(a, s.ws, SLOTS, ROWS);
    a.ctas = 2 * dev.num_sms;
    a.least = 1;
    a.unit_cost = 2.0f;
    CUtensorMap tk, tv;
    if (!attention_maps(kv, TILE, &tk, &tv)) return cudaErrorInvalidValue;
    return with_type(kv.type, [&](auto x) -> cudaError_t {
        using T = decltype(x);
        if constexpr (sizeof(T) == 4) {
            return cudaErrorInvalidValue;
        } else {
            auto go = [&](auto d) -> cudaError_t {
                constexpr int D = decltype(d)::value;
                constexpr size_t smem = 1024 + Cfg<D>::STAGES * Cfg<D>::STAGE_BYTES + sizeof(Shared);
                cudaError_t e = set_kernel_smem<attention_rows_kernel<T, D>>(dev.device, smem);
                if (e != cudaSuccess) return e;
                e = launch_dependent(attention_rows_kernel<T, D>, dim3(2 * dev.num_sms), THREADS, smem, stream, tk, tv, a);
                if (e != cudaSuccess) return e;
                return launch_dependent(attention_join_kernel<D, ROWS, TILE, COUNTERS, JOIN_WARPS>, dim3(4 * dev.num_sms), 32 * JOIN_WARPS, 0, stream, a);
            };
            return kv.dim == 64 ? go(std::integral_constant<int, 64>{}) : go(std::integral_constant<int, 128>{});
        }
    });
}

}  // namespace q8
