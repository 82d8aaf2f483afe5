// attention.cu -- causal attention of a few new tokens a sequence (one: decoding) over a paged cache.
//   s_j = scale q . k_j,  o = sum_j e^(s_j - mx) v_j / sum_j e^(s_j - mx)  over the visible positions j
//
// Bound by memory: each key and value is read once and serves the group's query heads.  All (row tile, 64
// positions) pairs of the batch stand in one line, and each CTA takes an equal stretch of it, so that 152 SMs
// are filled evenly whatever the number and the lengths of the sequences.  A row tile that a stretch cuts
// has parts in several CTAs, which attention_rows_join adds up.
//
// One warp brings 64 positions at a time to shared memory (TMA boxes of up to a page, 128-byte swizzled, several
// stages ahead across row tiles).  Four warps take 16 positions each, with their own running maximum and sum, so
// they meet only at the end of a row tile.  The products run on the warp-level tensor-core MMA: 16
// rows are too few for tcgen05's 128, and it is not what bounds.  Scores, statistics and sums are f32; the weights
// e^(s - mx) <= 1 are rounded to the cache's type for the second product, whose operands have one type
// (times a power of two, weight_shift).
//
// One token over 131071 positions of 32 + 8 heads x 128 bf16: 87 us (6.2 TB/s, 0.91 of a copy); 64 sequences of 500 to
// 8192: 108 us (0.91); 190 of 37 to 600, 12 heads x 64: 33.8 us (0.53: 7 us of launches, planning and joining kernel, the rest
// row tiles' ends: 7.5 a CTA, about 1.2 us each); one over 4096: 11 us (0.22: 6 us from launch to output, of which the first keys' way 2, then the
// joining kernel).
#include <algorithm>

#include "attention.cuh"

namespace q8 {
namespace {

constexpr int TILE = 64;             // positions a stage
constexpr int KEY_WARPS = 4;         // 16 positions each
constexpr int COUNTERS = 128;        // threads that count the work
constexpr float NEG = -INFINITY;

constexpr int ROWS = 16;              // of a row tile

template <int D>
struct Cfg {
    static constexpr int CTAS = 2;                              // to an SM
    static constexpr int THREADS = 32 * (KEY_WARPS + 1);
    static constexpr int TILE_BYTES = TILE * D * 2;             // of keys, and of values
    static constexpr int STAGE_BYTES = 2 * TILE_BYTES;
    static constexpr int STAGES = 96 * 1024 / STAGE_BYTES;
    static constexpr int HALVES = D / 64;                       // 128-byte wide columns of a tile
    static constexpr int Q_STRIDE = D * 2 + 16;                 // bytes: rows in different banks
    static constexpr int Q_BYTES = ROWS * Q_STRIDE, Q_BUFFERS = 3;
    static constexpr int OFF_Q = STAGES * STAGE_BYTES, OFF_SHARED = OFF_Q + Q_BUFFERS * Q_BYTES;
};

struct Shared {
    long long before[COUNTERS + 1];       // work before thread j's sequences
    long long sums[COUNTERS / 32];
    uint64_t full[6], empty[6], q_full[3], q_empty[3];
    uint32_t ok[6];                       // a stage's 16-position blocks whose page exists
    float mx[2][KEY_WARPS][ROWS], sum[2][KEY_WARPS][ROWS];
    int spoilt[2][KEY_WARPS];             // a non-finite value that some rows see has been cleared
    int abort_flag;
};

// ---------------------------------------------------------------------------------------
// The line of work: the sequences one after another, in each the row tiles and in these the heads, each with
// the key tiles that its longest row tile sees (one at least, so that rows that see nothing are written too) behind
// `extra` that stand for what a row tile costs beside them.  A stretch that ends among the latter has nothing of
// the row tile, and one that begins there has all of its beginning.
// ---------------------------------------------------------------------------------------
// 64-bit division, mostly of numbers that fit 32 bits.
__device__ __forceinline__ long long divide(long long x, long long by)
{
    return ((x | by) >> 32) == 0 ? (long long)((uint32_t)x / (uint32_t)by) : x / by;
}

struct Line {
    long long total, length;      // key tiles, and of a CTA's stretch
    // Up to 32 sequences: each lane of each warp has one, and the work before it.  More: counting thread j has `per`.
    bool few;
    int per;
    long long before;
    int items, n;
    Seq s;

    // Row tiles x heads of a sequence, and key tiles of each.
    static __device__ __forceinline__ void shape(const Attn &a, const Seq &s, int &items, int &n)
    {
        const int rows = s.n * a.group, tiles = (rows + ROWS - 1) / ROWS;
        items = tiles * a.p.heads;
        n = 0;
        if (!tiles) return;
        n = span_of<TILE>(a, s, (tiles - 1) * ROWS, rows - 1).n;
        if (tiles > 1 && a.window) {        // another row tile's window may touch one tile more
            const int tokens = a.by_group(ROWS + a.group - 2) + 1;
            n = min(min(s.pos0 + s.n, s.end), 0x3fffffff) / TILE + 1;
            n = min(n, (int)((a.window + (long long)tokens + TILE - 3) / TILE) + 1);
        }
        n = max(n, 1) + a.extra;
    }

    // Called by all threads of the CTA.  (Few sequences: no barrier.)
    __device__ __forceinline__ void make(const Attn &a, long long *starts, long long *sums)
    {
        const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
        few = a.p.seqs <= 32;
        per = (a.p.seqs + COUNTERS - 1) / COUNTERS;
        items = n = 0;
        long long w = 0;
        if (few) {
            if (lane < a.p.seqs) {
                s = seq_of(a.p, lane);
                shape(a, s, items, n);
                w = (long long)items * n;
            }
        } else if (t < COUNTERS) {
            for (int b = t * per; b < min(t * per + per, a.p.seqs); ++b) {
                int i, k;
                shape(a, seq_of(a.p, b), i, k);
                w += (long long)i * k;
            }
        }
        long long sum = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += u;
        }
        if (few) {
            before = sum - w;
            total = __shfl_sync(0xffffffffu, sum, 31);
        } else {
            if (t < COUNTERS && lane == 31) sums[warp] = sum;
            __syncthreads();
            if (t < COUNTERS) {
#pragma unroll
                for (int j = 0; j < COUNTERS / 32; ++j)
                    if (j < warp) sum += sums[j];
                starts[t] = sum - w;
                if (t == COUNTERS - 1) starts[COUNTERS] = sum;
            }
            __syncthreads();
            total = starts[COUNTERS];
        }
        length = max(divide(total + a.ctas - 1, a.ctas), (long long)a.least);
    }
};

// A place on the line.  Its calls are made by whole warps.
struct Place {
    int b, item, items, n, tile;       // sequence, row tile and head of so many, key tile of so many (extra ones included)
    Seq s;

    __device__ __forceinline__ void enter(const Attn &a, const Line &line)
    {
        if (line.few) {
            items = __shfl_sync(0xffffffffu, line.items, b);
            n = __shfl_sync(0xffffffffu, line.n, b);
            s.row0 = __shfl_sync(0xffffffffu, line.s.row0, b);
            s.n = __shfl_sync(0xffffffffu, line.s.n, b);
            s.pos0 = __shfl_sync(0xffffffffu, line.s.pos0, b);
            s.end = __shfl_sync(0xffffffffu, line.s.end, b);
        } else {
            s = seq_of(a.p, b);
            Line::shape(a, s, items, n);
        }
    }
    // Key tile x of the line (x < total).
    __device__ __forceinline__ Place(const Attn &a, const Line &line, const long long *starts, long long x)
    {
        long long left;
        if (line.few) {
            b = __popc(__ballot_sync(0xffffffffu, line.before <= x)) - 1;    // (those behind the last hold the total)
            left = x - __shfl_sync(0xffffffffu, line.before, b);
            enter(a, line);
        } else {
            int lo = -1;                   // the last thread that starts at or before x
#pragma unroll
            for (int i = 0; i < COUNTERS; i += 32) lo += __popc(__ballot_sync(0xffffffffu, starts[i + (threadIdx.x & 31)] <= x));
            left = x - starts[lo];
            for (b = lo * line.per;; ++b) {
                enter(a, line);
                if (left < (long long)items * n || b + 1 >= a.p.seqs) break;
                left -= (long long)items * n;
            }
        }
        item = n ? (int)divide(left, n) : 0;
        tile = (int)(left - (long long)item * n);
    }
    // The next row tile's first key tile (not behind the line's end).
    __device__ __forceinline__ void next(const Attn &a, const Line &line)
    {
        tile = 0;
        if (++item < items) return;
        item = 0;
        do {
            if (++b >= a.p.seqs) return;
            enter(a, line);
        } while (items == 0);
    }
};

// The part of a row tile that a CTA's stretch holds.
struct Part {
    int h, r0, valid;                  // head of keys and values; first row and how many
    int t0, t1;                        // key tiles
    Span span;
    bool whole;

    __device__ __forceinline__ Part(const Attn &a, const Place &p, long long left)
    {
        const int tile = a.by_heads(p.item), end = (int)min((long long)p.n, p.tile + left);      // end > extra
        h = p.item - tile * a.p.heads;
        r0 = tile * ROWS;
        valid = min(ROWS, p.s.n * a.group - r0);
        span = span_of<TILE>(a, p.s, r0, r0 + valid - 1);
        t0 = span.first + min(max(p.tile - a.extra, 0), span.n);
        t1 = span.first + min(end - a.extra, span.n);
        whole = p.tile == 0 && end == p.n;
    }
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

// A word's halves, zeros in place of infinities and NaN.
template <typename T>
__device__ __forceinline__ uint32_t finite2(uint32_t w)
{
    constexpr uint32_t E = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
    return w & ((w & E) == E ? 0xffff0000u : ~0u) & ((w >> 16 & E) == E ? 0x0000ffffu : ~0u);
}

// A warp's 16 positions of a tile of values: cleared outside lo .. hi, and inside where not finite; whether something
// was (in this lane's part).  (128-byte rows swizzle within themselves, so where a value stands does not matter.)
template <typename T, int D>
__device__ __forceinline__ bool clear_block(uint8_t *values, int lo, int hi)
{
    constexpr int VECS = D / 8;                     // 16-byte vectors of a position
    const int lane = threadIdx.x & 31, v = lane % VECS;
    uint8_t *p = values + (v >> 3) * (TILE * 128) + (v & 7) * 16;
    bool found = false;
#pragma unroll
    for (int r = lane / VECS; r < 16; r += 32 / VECS) {
        uint4 *w = reinterpret_cast<uint4 *>(p + r * 128), u = *w;
        if (r < lo || r > hi) {
            u = make_uint4(0, 0, 0, 0);
            *w = u;
        }
        const uint4 f = make_uint4(finite2<T>(u.x), finite2<T>(u.y), finite2<T>(u.z), finite2<T>(u.w));
        if (f.x != u.x || f.y != u.y || f.z != u.z || f.w != u.w) {
            found = true;
            *w = f;
        }
    }
    __syncwarp();
    return found;
}

template <typename T, int D>
__global__ void __launch_bounds__(Cfg<D>::THREADS, Cfg<D>::CTAS)
    attention_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, Attn a)
{
    using C = Cfg<D>;
    extern __shared__ __align__(1024) uint8_t stages[];
    Shared &sm = *reinterpret_cast<Shared *>(stages + C::OFF_SHARED);
    volatile int *abort_flag = &sm.abort_flag;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) { mbar_init(&sm.full[s], 1); mbar_init(&sm.empty[s], KEY_WARPS); }
        for (int s = 0; s < C::Q_BUFFERS; ++s) { mbar_init(&sm.q_full[s], 1); mbar_init(&sm.q_empty[s], KEY_WARPS); }
        sm.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == KEY_WARPS && lane == 0) {
        prefetch_tensormap(&tm_k);
        prefetch_tensormap(&tm_v);
    }
    griddep_wait();
    griddep_launch_dependents();
    Line line{};
    line.make(a, sm.before, sm.sums);
    __syncthreads();                                             // the barriers exist for all
    long long x = blockIdx.x * line.length;
    const long long x1 = min(x + line.length, line.total);
    if (x >= x1) return;
    Place place(a, line, sm.before, x);
    if (place.tile <= a.extra) {
        x -= place.tile;
        place.tile = 0;
    }
    auto more = [&] { return x < x1 && place.tile + (x1 - x) > a.extra; };

    if (warp == KEY_WARPS) {
        // ------------------------------ producer ------------------------------
        const int ps = 1 << a.p.page_shift, per_tile = ps < TILE ? TILE / ps : 1, blocks = 4 / per_tile;
        int it = 0, st = 0, parts = 0;
        uint32_t phase = 1;
        bool ok = true;
        for (; ok && more(); ++parts) {
            const Part p(a, place, x1 - x);
            const Seq s = place.s;
            const int b = place.b;
            x += min((long long)(place.n - place.tile), x1 - x);
            place.next(a, line);
            // (on its way while the queries' copies are set up, as the next tile's is while this one's are)
            int64_t page = lane < per_tile && p.t0 < p.t1 ? page_of(a.p, b, (p.t0 * TILE >> a.p.page_shift) + lane) : -1;
            // Queries, a row a lane (rows behind the last one hold anything: what comes of them goes nowhere).
            const int qb = parts % C::Q_BUFFERS;
            ok = __all_sync(0xffffffffu, wait_or_abort(&sm.q_empty[qb], (parts / C::Q_BUFFERS & 1) ^ 1, a.status, abort_flag));
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(&sm.q_full[qb], p.valid * D * 2);
            __syncwarp();
            for (int i = lane; i < p.valid; i += 32) {
                const int r = p.r0 + i, tok = a.by_group(r);
                bulk_g2s(stages + C::OFF_Q + qb * C::Q_BYTES + i * C::Q_STRIDE,
                         static_cast<const T *>(a.q) + (s.row0 + tok) * a.ldq + (p.h * a.group + r - tok * a.group) * D, D * 2,
                         &sm.q_full[qb]);
            }
            __syncwarp();
            for (int t = p.t0; t < p.t1; ++t, ++it) {
                const int pos = t * TILE;
                const uint32_t good = __ballot_sync(0xffffffffu, page >= 0);
                uint32_t okm = 0;
                for (int j = 0; j < per_tile; ++j)
                    if (good >> j & 1) okm |= ((1u << blocks) - 1) << (j * blocks);
                // A page that does not exist: a box outside the tensor, which reads as zeros.
                const int id = page < 0 ? (int)a.p.pages : (int)page;
                if (t + 1 < p.t1 && lane < per_tile) page = page_of(a.p, b, ((pos + TILE) >> a.p.page_shift) + lane);
                ok = __all_sync(0xffffffffu, wait_or_abort(&sm.empty[st], phase, a.status, abort_flag));
                if (!ok) break;
                if (lane == 0) {
                    sm.ok[st] = okm;
                    mbar_arrive_expect_tx(&sm.full[st], C::STAGE_BYTES);
                }
                __syncwarp();
                const int j = lane / (2 * C::HALVES), half = lane % C::HALVES, is_v = lane / C::HALVES % 2;
                const int box_page = __shfl_sync(0xffffffffu, id, j);
                if (j < per_tile)
                    tma_load_4d(stages + st * C::STAGE_BYTES + is_v * C::TILE_BYTES + half * (TILE * 128) + j * ps * 128,
                                is_v ? &tm_v : &tm_k, half * 64, ps > TILE ? pos & (ps - 1) : 0, p.h, box_page, &sm.full[st]);
                if (++st == C::STAGES) {
                    st = 0;
                    phase ^= 1;
                }
            }
        }
        // Never leave with a copy into this CTA's shared memory in flight.
        for (int i = it > C::STAGES ? it - C::STAGES : 0; i < it; ++i)
            mbar_wait_drain(&sm.full[i % C::STAGES], (i / C::STAGES) & 1, a.status);
        for (int i = max(parts - C::Q_BUFFERS, 0); i < parts; ++i)
            mbar_wait_drain(&sm.q_full[i % C::Q_BUFFERS], i / C::Q_BUFFERS & 1, a.status);
        return;
    }

    // ------------------------------ consumers ------------------------------
    const int g = lane >> 2, c = lane & 3, kw = warp;
    const uint32_t stage0 = smem_u32(stages);
    // Rows of this lane's ldmatrix addresses: queries, keys in their own order, values transposed.
    const uint32_t q0 = stage0 + C::OFF_Q + ((lane & 7) + (lane >> 3 & 1) * 8) * C::Q_STRIDE + (lane >> 4) * 16;
    const int krow = kw * 16 + (lane & 7) + (lane >> 4) * 8, kchunk = lane >> 3 & 1;
    const int vrow = kw * 16 + (lane & 7) + (lane >> 3 & 1) * 8, vchunk = lane >> 4;
    const long long x0 = x;
    int st = 0;
    uint32_t phase = 0;
    for (int parts = 0; more(); ++parts) {
        const Part p(a, place, x1 - x);
        const Seq s0 = place.s;
        const int b = place.b, flip = parts & 1, qb = parts % C::Q_BUFFERS;
        const int slot = p.whole ? -1 : 2 * (int)blockIdx.x + (x != x0);
        x += min((long long)(place.n - place.tile), x1 - x);
        place.next(a, line);
        const int first = s0.pos0 + a.by_group(p.r0), last = s0.pos0 + a.by_group(p.r0 + p.valid - 1);    // positions of its rows

        // Two rows a lane: g and g + 8.
        int lo[2], hi[2];
        float o[D / 8][4], mx[2], sum[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = g + 8 * i, pos = s0.pos0 + a.by_group(p.r0 + r);
            hi[i] = r < p.valid ? min(pos, s0.end - 1) : -1;
            lo[i] = a.window ? max(pos - a.window + 1, 0) : 0;
            mx[i] = NEG;
            sum[i] = 0.0f;
        }
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[n][i] = 0.0f;
        bool spoilt = false;
        bool aborted = !__all_sync(0xffffffffu, wait_or_abort(&sm.q_full[qb], parts / C::Q_BUFFERS & 1, a.status, abort_flag));
        const uint32_t qs = q0 + qb * C::Q_BYTES;
        uint32_t q[D / 16][4];
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) ldmatrix_x4(q[kk], qs + kk * 32);

        for (int t = p.t0; t < p.t1; ++t) {
            if (!aborted) aborted = !__all_sync(0xffffffffu, wait_or_abort(&sm.full[st], phase, a.status, abort_flag));
            if (aborted) break;
            const uint32_t kt = stage0 + st * C::STAGE_BYTES, vt = kt + C::TILE_BYTES;
            const int key0 = t * TILE + kw * 16;
            // The warp's 16 positions, unless no row sees one.
            if ((sm.ok[st] >> kw & 1) && key0 <= p.span.hi && key0 + 15 >= p.span.lo) {
                // Columns of s[n]: positions key0 + 8 n + 2 c and the next; rows g (0, 1) and g + 8 (2, 3).
                float s[2][4] = {};
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    uint32_t kf[4];
                    const int chunk = kk * 2 + kchunk;
                    ldmatrix_x4(kf, kt + (chunk >> 3) * (TILE * 128) + krow * 128 + (((chunk & 7) ^ (krow & 7)) << 4));
                    mma_16816<T>(s[0], q[kk], kf[0], kf[1]);
                    mma_16816<T>(s[1], q[kk], kf[2], kf[3]);
                }
                // Some row does not see some of them.
                if (key0 < p.span.lo || key0 + 15 > min(first, p.span.hi) || (a.window && key0 <= last - a.window)) {
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int key = key0 + 8 * n + 2 * c + (i & 1);
                            if (key < lo[i >> 1] || key > hi[i >> 1]) s[n][i] = NEG;
                        }
                    spoilt |= clear_block<T, D>(stages + (vt - stage0) + kw * (16 * 128), p.span.lo - key0, p.span.hi - key0);
                }
                uint32_t pf[4];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    // Products rounded before mx is subtracted: the largest score's exponent is within the shift whatever its size,
                    // where an fma's would be what the product in mx has been rounded by.
                    float e[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) e[j] = __fmul_rn(s[j >> 1][2 * i + (j & 1)], a.scale);
                    float m = fmaxf(fmaxf(e[0], e[1]), fmaxf(e[2], e[3]));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
                    m = fmaxf(mx[i], shifted<T>(m, 1.0f, 0));
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
#pragma unroll
                    for (int j = 0; j < 4; ++j) e[j] = attn_ex2(__fsub_rn(e[j], base));
                    sum[i] += (e[0] + e[1]) + (e[2] + e[3]);
                    pf[i] = pack2<T>(e[0], e[1]);
                    pf[i + 2] = pack2<T>(e[2], e[3]);
                }
#pragma unroll
                for (int n = 0; n < D / 16; ++n) {
                    uint32_t vf[4];
                    const int chunk = 2 * n + vchunk;
                    ldmatrix_x4_trans(vf, vt + (chunk >> 3) * (TILE * 128) + vrow * 128 + (((chunk & 7) ^ (vrow & 7)) << 4));
                    mma_16816<T>(o[2 * n], pf, vf[0], vf[1]);
                    mma_16816<T>(o[2 * n + 1], pf, vf[2], vf[3]);
                }
            }
            // The last stage is handed back after the join, which uses its memory.
            if (t + 1 < p.t1) {
                fence_proxy_async_smem();                // reads before the next copies to the stage
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.empty[st]);
                if (++st == C::STAGES) {
                    st = 0;
                    phase ^= 1;
                }
            }
        }

        // ---- join of the four warps with the same rows ----
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
            sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
            if (c == 0) {
                sm.mx[flip][kw][g + 8 * i] = mx[i];
                sm.sum[flip][kw][g + 8 * i] = sum[i];
            }
        }
        spoilt = __any_sync(0xffffffffu, spoilt);
        if (lane == 0) sm.spoilt[flip][warp] = spoilt;
        // (the next part's words go to the other flip: some warps may still read these.  They are written again only
        // behind the next part's barrier)
        // The queries are handed back behind this barrier, where what has become of them has been exchanged.  (An arrival right
        // behind their loads passed these where another CTA's filled the load queue, and the next queries came in between: of 10000
        // sequences three rows a call.)
        fence_proxy_async_smem();
        if (bar_red_or(1, 32 * KEY_WARPS, aborted)) return;
        if (lane == 0) mbar_arrive(&sm.q_empty[qb]);
        const bool some = p.t1 > p.t0;
        float *join = reinterpret_cast<float *>(stages + st * C::STAGE_BYTES);      // [warp][row][D], 16-byte words swizzled by row
        if (some) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = g + 8 * i;
                float m = NEG;
#pragma unroll
                for (int w = 0; w < KEY_WARPS; ++w) m = fmaxf(m, sm.mx[flip][w][r]);
                const float f = attn_ex2(mx[i] - (m == NEG ? 0.0f : m));
#pragma unroll
                for (int n = 0; n < D / 8; ++n) {
                    const int col = (8 * n + 2 * c) ^ ((r & 7) << 2);
                    *reinterpret_cast<float2 *>(join + (kw * 16 + r) * D + col) = make_float2(o[n][2 * i] * f, o[n][2 * i + 1] * f);
                }
            }
            named_bar_sync(2, 32 * KEY_WARPS);
        }
        const int r = (threadIdx.x >> 3) & 15, c8 = threadIdx.x & 7;        // a row, and every eighth vector of it
        if (r < p.valid) {
            float m = NEG, l = 0.0f;
#pragma unroll
            for (int w = 0; w < KEY_WARPS; ++w) m = fmaxf(m, sm.mx[flip][w][r]);
            const float base = m == NEG ? 0.0f : m;
#pragma unroll
            for (int w = 0; w < KEY_WARPS; ++w) l += sm.sum[flip][w][r] * attn_ex2(sm.mx[flip][w][r] - base);
            float acc[D / 8];
#pragma unroll
            for (int j = 0; j < D / 8; ++j) acc[j] = 0.0f;
            if (some) {
#pragma unroll
                for (int w = 0; w < KEY_WARPS; ++w)
#pragma unroll
                    for (int j = 0; j < D / 32; ++j) {
                        const float4 v = *reinterpret_cast<const float4 *>(
                            join + (w * 16 + r) * D + (((j * 8 + c8) ^ (r & 7)) << 2));
                        acc[4 * j] += v.x;
                        acc[4 * j + 1] += v.y;
                        acc[4 * j + 2] += v.z;
                        acc[4 * j + 3] += v.w;
                    }
            }
            const int row = p.r0 + r, tok = a.by_group(row), head = p.h * a.group + row - tok * a.group;
            int sp = 0;
#pragma unroll
            for (int w = 0; w < KEY_WARPS; ++w) sp |= sm.spoilt[flip][w];
            if (sp) {
                const int pos = s0.pos0 + tok;
                const int k0 = max(a.window ? pos - a.window + 1 : 0, p.t0 * TILE), k1 = min(min(pos, s0.end - 1), p.t1 * TILE - 1);
                float e[D / 8];
                for (int j = 0; j < D / 8; ++j) e[j] = 0.0f;
                const T *qr = static_cast<const T *>(a.q) + (s0.row0 + tok) * a.ldq + head * D;
                auto col = [&](int j) { return ((j >> 2) * 8 + c8) * 4 + (j & 3); };
                // The blocks of 16 that were taken as not seen by all rows.
                if (a.window) add_non_finite<T, D>(a, b, p.h, qr, k0, min(k1, (last - a.window) | 15), base, col, e);
                add_non_finite<T, D>(a, b, p.h, qr, max(k0, (min(first, p.span.hi) + 1) & ~15), k1, base, col, e);
#pragma unroll
                for (int j = 0; j < D / 8; ++j) acc[j] += e[j];
            }
            if (slot >= 0) {
                const int64_t at = (int64_t)slot * ROWS + r;
                if (c8 == 0) a.ml[at] = make_float2(m, l);
#pragma unroll
                for (int j = 0; j < D / 32; ++j)
                    *reinterpret_cast<float4 *>(a.part + at * D + (j * 8 + c8) * 4) =
                        make_float4(acc[4 * j], acc[4 * j + 1], acc[4 * j + 2], acc[4 * j + 3]);
            } else {
                const float inv = l == 0.0f ? 0.0f : 1.0f / l;       // a row that sees nothing: 0
                uint8_t *dst = static_cast<uint8_t *>(a.out) +
                               ((s0.row0 + tok) * a.ldo + head * D) * out_size(a.otype);
#pragma unroll
                for (int j = 0; j < D / 32; ++j)
                    store4(dst + (j * 8 + c8) * 4 * out_size(a.otype), a.otype,
                           make_float4(acc[4 * j] * inv, acc[4 * j + 1] * inv, acc[4 * j + 2] * inv, acc[4 * j + 3] * inv));
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
    }
}

constexpr int JOIN_WARPS = 4, JOIN_Y = 4;

// A row's parts, added in their order by four warps: o = sum_i e^(mx_i - mx) o_i / sum_i e^(mx_i - mx) sum_i.  A
// warp takes its parts relative to its own maximum, eight loads at a time.  slot(i): where part i is.
template <int D, typename Slot>
__device__ __forceinline__ void join_row(const Attn &a, int parts, Slot slot, int r, uint8_t *dst, float (&acc)[JOIN_WARPS][D],
                                         float (&mw)[JOIN_WARPS], float (&lw)[JOIN_WARPS])
{
    constexpr int V = D / 32, U = 8;         // values a lane, parts at a time
    using Vec = std::conditional_t<V == 4, float4, float2>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int s0 = parts * warp / JOIN_WARPS, s1 = parts * (warp + 1) / JOIN_WARPS;
    float m = NEG, l = 0.0f, v[V] = {};
    for (int s = s0; s < s1; s += U) {
        float2 ml[U];
        Vec w[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int64_t at = (int64_t)slot(min(s + i, s1 - 1)) * ROWS + r;
            ml[i] = a.ml[at];
            w[i] = *reinterpret_cast<const Vec *>(a.part + at * D + V * lane);
        }
        float top = m;
#pragma unroll
        for (int i = 0; i < U; ++i) top = fmaxf(top, ml[i].x);
        const float base = top == NEG ? 0.0f : top, f0 = attn_ex2(m - base);
        m = top;
        l *= f0;
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] *= f0;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (s + i >= s1) break;
            const float f = attn_ex2(ml[i].x - base);
            l = fmaf(ml[i].y, f, l);
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] = fmaf(reinterpret_cast<const float *>(&w[i])[j], f, v[j]);
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) acc[warp][V * lane + j] = v[j];
    if (lane == 0) {
        mw[warp] = m;
        lw[warp] = l;
    }
    __syncthreads();
    if (threadIdx.x < D / 4) {
        float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        m = NEG;
        l = 0.0f;
#pragma unroll
        for (int w = 0; w < JOIN_WARPS; ++w) m = fmaxf(m, mw[w]);
        const float base = m == NEG ? 0.0f : m;
#pragma unroll
        for (int w = 0; w < JOIN_WARPS; ++w) {
            const float4 u = *reinterpret_cast<const float4 *>(&acc[w][4 * threadIdx.x]);
            const float f = attn_ex2(mw[w] - base);
            t.x = fmaf(u.x, f, t.x);
            t.y = fmaf(u.y, f, t.y);
            t.z = fmaf(u.z, f, t.z);
            t.w = fmaf(u.w, f, t.w);
            l = fmaf(lw[w], f, l);
        }
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        store4(dst + 4 * threadIdx.x * out_size(a.otype), a.otype, make_float4(t.x * inv, t.y * inv, t.z * inv, t.w * inv));
    }
    __syncthreads();
}

// CTA (c, y) joins the row tile that the end of stretch c cuts first, rows y, y + 4, ...  It works out which one while
// the parts are still being computed (what starts and lens hold was there before the kernel in front, which
// has waited for it).
template <int D>
__global__ void __launch_bounds__(32 * JOIN_WARPS) attention_rows_join_kernel(Attn a)
{
    __shared__ long long before[COUNTERS + 1], sums[COUNTERS / 32];
    __shared__ alignas(16) float acc[JOIN_WARPS][D];
    __shared__ float mw[JOIN_WARPS], lw[JOIN_WARPS];
    Line line{};
    line.make(a, before, sums);
    const long long len = line.length, x = (blockIdx.x + 1) * len;
    if (x < line.total) {
        const Place p(a, line, before, x);
        const long long start = x - p.tile;                  // of the row tile
        if (p.tile > a.extra && x - len - start <= a.extra) {
            const int k0 = blockIdx.x, parts = (int)divide(start + p.n - 1, len) - k0 + 1;
            const int tile = a.by_heads(p.item), h = p.item - tile * a.p.heads, valid = min(ROWS, p.s.n * a.group - tile * ROWS);
            griddep_wait();
            for (int r = blockIdx.y; r < valid; r += JOIN_Y) {
                const int row = tile * ROWS + r, tok = a.by_group(row), head = h * a.group + row - tok * a.group;
                // Its first part is its stretch's last one, unless the stretch begins with it; the others are first.
                join_row<D>(a, parts, [&](int i) { return 2 * (k0 + i) + (i == 0 && x - len < start); }, r,
                                  static_cast<uint8_t *>(a.out) + ((p.s.row0 + tok) * a.ldo + head * D) * out_size(a.otype), acc, mw, lw);
            }
        }
    }
    griddep_enter();
}

// ---------------------------------------------------------------------------------------
// The same for row tiles of chunks, which have many rows in few parts: a row a warp, as many consecutive ones as there
// are more rows than warps.  Latency: what finds the rows ran ahead, then one load's time a row (2240 rows of seven parts at
// most 10 us -> 4 by spreading the rows that exist; 16384 rows of two parts 5 us, two rows at a time the same).
// ---------------------------------------------------------------------------------------
constexpr int CHUNK_JOIN_THREADS = 256;

template <int D, bool FEW>
__global__ void __launch_bounds__(CHUNK_JOIN_THREADS) attention_chunk_join_kernel(Attn a)
{
    constexpr int V = D / 32, U = 4;             // values a lane, parts at a time
    using Vec = std::conditional_t<V == 4, float4, float2>;
    const int lane = threadIdx.x & 31, warps = gridDim.x * (CHUNK_JOIN_THREADS / 32);
    using P = Plan<CHUNK_ROWS, CHUNK_TILE, FEW>;
    __shared__ P plans[32];                      // one warp's, for all
    if (threadIdx.x < 32) {
        P p;
        p.make(a);
        plans[lane] = p;
    }
    __syncthreads();
    const P plan = plans[lane];
    const int each = (plan.split + warps - 1) / warps;
    int i = (blockIdx.x * (CHUNK_JOIN_THREADS / 32) + (threadIdx.x >> 5)) * each;
    const int end = min(i + each, plan.split);
    Unit x;
    int row = 0, left = 0;                       // of the sequence and head; how many more
    if (i < end) {
        x = plan.find_row(a, i, row);
        left = x.s.n * a.group - row;
    }
    griddep_enter();
    for (; i < end; ++i, ++row, --left) {
        if (!left) {
            x = plan.find_row(a, i, row);
            left = x.s.n * a.group - row;
        }
        const int tile = row / CHUNK_ROWS;
        const int64_t at = (int64_t)(x.slot + ((x.tile - 1 - tile) * a.p.heads + x.h) * x.parts) * CHUNK_ROWS + (row - tile * CHUNK_ROWS);
        float m = NEG, l = 0.0f, v[V] = {};
        for (int s = 0; s < x.parts; s += U) {
            float2 ml[U];
            Vec w[U];
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const int64_t p = at + (int64_t)min(s + k, x.parts - 1) * CHUNK_ROWS;
                ml[k] = a.ml[p];
                w[k] = *reinterpret_cast<const Vec *>(a.part + p * D + V * lane);
            }
            float top = m;
#pragma unroll
            for (int k = 0; k < U; ++k) top = fmaxf(top, ml[k].x);
            const float base = top == NEG ? 0.0f : top, f0 = attn_ex2(m - base);
            m = top;
            l *= f0;
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] *= f0;
#pragma unroll
            for (int k = 0; k < U; ++k) {
                if (s + k >= x.parts) break;
                const float f = attn_ex2(ml[k].x - base);
                l = fmaf(ml[k].y, f, l);
#pragma unroll
                for (int j = 0; j < V; ++j) v[j] = fmaf(reinterpret_cast<const float *>(&w[k])[j], f, v[j]);
            }
        }
        const int tok = a.by_group(row), head = x.h * a.group + row - tok * a.group;
        uint8_t *dst = static_cast<uint8_t *>(a.out) + ((x.s.row0 + tok) * a.ldo + head * D) * out_size(a.otype);
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        if constexpr (V == 4) {
            store4(dst + 4 * lane * out_size(a.otype), a.otype, make_float4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv));
        } else {
            const float y = __shfl_down_sync(0xffffffffu, v[0] * inv, 1), z = __shfl_down_sync(0xffffffffu, v[1] * inv, 1);
            if (!(lane & 1)) store4(dst + 2 * lane * out_size(a.otype), a.otype, make_float4(v[0] * inv, v[1] * inv, y, z));
        }
    }
}

}  // namespace

cudaError_t launch_attention_chunk_join(const DeviceInfo &dev, const Attn &a, int dim, cudaStream_t stream)
{
    auto go = [&](auto kern) { return launch_dependent(kern, dim3(4 * dev.num_sms), CHUNK_JOIN_THREADS, 0, stream, a); };
    if (a.p.seqs <= 32) return dim == 64 ? go(attention_chunk_join_kernel<64, true>) : go(attention_chunk_join_kernel<128, true>);
    return dim == 64 ? go(attention_chunk_join_kernel<64, false>) : go(attention_chunk_join_kernel<128, false>);
}

// Enough for either kernel: of few rows, two partial results at most of each of the two CTAs on each of 152 SMs.
size_t attention_workspace_bytes(int dim) { return std::max(attention_space(2 * 2 * 152, ROWS, dim), attention_chunk_space(dim)); }

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
    a.far_scale = exp2f(floorf(log2f(a.scale)) + 1.0f);
    a.status = dev.status;
    const int64_t most = s.max_new && s.max_new < m ? s.max_new : m;     // new tokens of a sequence
    // One row tile of 16 a head here, or half full ones of 256 there: 16 sequences at 6000 of 28 + 4 heads x 128, 14
    // rows 43 us here and 56 there; 100 at 1000 of 64 + 8 heads x 64, 16 rows 47 and 67; one at 6000, 14 rows 22 and
    // 29.  From 17 rows on a sequence's keys would be read and multiplied for two row tiles here: two row tiles side
    // by side in registers took 54 us for 57 there at 21 rows of the first, but 33 for 29 of the last, and at 28 to 32
    // rows up to a third more (16 at 600 24 us, there 17).
    if (most * a.group > ROWS) return launch_attention_chunk(dev, kv, a, s.ws, stream);
    CUtensorMap tk, tv;
    if (!attention_maps(kv, TILE, &tk, &tv)) return cudaErrorInvalidValue;
    return with_type(kv.type, [&](auto x) -> cudaError_t {
        using T = decltype(x);
        if constexpr (sizeof(T) == 4) {
            return cudaErrorInvalidValue;
        } else {
            auto go = [&](auto d) -> cudaError_t {
                constexpr int D = decltype(d)::value;
                using C = Cfg<D>;
                constexpr size_t smem = C::OFF_SHARED + sizeof(Shared);
                static_assert(smem <= 113 * 1024, "two CTAs to an SM");
                a.ctas = C::CTAS * std::min(dev.num_sms, 152);
                a.least = 2;
                a.extra = 2;             // (190 of 37 to 600, 12 heads x 64: none 46 us, 1 36, 2 33, 3 34; longer ones the same)
                attention_place(a, s.ws, 2 * a.ctas, ROWS);
                cudaError_t e = set_kernel_smem<attention_rows_kernel<T, D>>(dev.device, smem);
                if (e != cudaSuccess) return e;
                e = launch_dependent(attention_rows_kernel<T, D>, dim3(a.ctas), C::THREADS, smem, stream, tk, tv, a);
                if (e != cudaSuccess) return e;
                return launch_dependent(attention_rows_join_kernel<D>, dim3(a.ctas - 1, JOIN_Y), 32 * JOIN_WARPS, 0, stream, a);
            };
            return kv.dim == 64 ? go(std::integral_constant<int, 64>{}) : go(std::integral_constant<int, 128>{});
        }
    });
}

}  // namespace q8
