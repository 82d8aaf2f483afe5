// attention.cuh -- what the attention kernels share: how a batch is cut into units of work, masks,
// the way round non-finite values, partial results and output.
//
// Rows: the query heads that share a key/value head are rows of one matrix, row r of a sequence being
// query head r % group of its new token r / group; ROWS consecutive rows are a row tile.  A row tile's
// visible positions, in key tiles of TILE, are cut into `parts` so that the whole batch fills the GPU; a
// unit is one part.  Everything follows from starts and lens on the device, which a captured graph may
// find changed at each replay.
#pragma once

#include <cuda_bf16.h>
#include <limits.h>

#include "launch.h"
#include "paged.cuh"
#include "tcgen05.cuh"
#include "types.cuh"

namespace q8 {

// Division of 0 .. 2^31 - 1 by a number that the launch fixes.
struct Divide {
    uint32_t factor, shift = 0;
    Divide(uint32_t d = 1)
    {
        while ((1u << shift) < d) ++shift;
        factor = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << shift) - d)) / d + 1);
    }
    __device__ __forceinline__ int operator()(int n) const { return (int)((__umulhi(factor, (uint32_t)n) + (uint32_t)n) >> shift); }
};

struct Attn {
    Paged p;
    Divide by_group, by_heads;
    const void *kc, *vc, *q;
    void *out;
    int64_t ldq, ldo;
    int group, otype, window;    // window 0: all earlier positions
    float scale;                 // of scores, times log2 e
    float far_scale;             // the next power of two above it (attention_tc.cu)
    // How units are cut (Plan): CTAs that take them, the fewest key tiles that a part is worth, what a unit costs beside
    // its tiles (in tiles), partial results that the workspace has room for.
    int ctas, least, slots;
    float unit_cost;
    int extra;                   // (few rows) what a row tile costs beside its key tiles, in these
    // partial results of row tiles in several parts (attention_workspace)
    float2 *ml;                  // [slot][ROWS]: running maximum and sum
    float *part;                 // [slot][ROWS][D]
    int *status;
};

__device__ __forceinline__ float attn_ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// The weights 2^(s scale - mx) are rounded to T for the second product, and mx is not the largest score itself but `shift` below it;
// lag: by how much a score may pass the largest one that mx knows of.
// f16 ends at 2^-24: weights reach up to 2^15, so that they fill the type's range and many small ones are not lost beside a large one.
// bf16 has the range in its values, too: weights stay below 2^-20, so that the sum of a million of the largest values is still
// within f32 before it is divided (and values down to 2^-100 keep their precision there).
template <typename T>
__device__ constexpr float weight_shift(int lag) { return (std::is_same<T, __half>::value ? 15 : -20) - lag; }
// mx of the largest score's product with its scale: rounded towards that product, so that the weight is not beyond 1 and 2^shift
// however far apart the numbers of f32 are there.
template <typename T>
__device__ __forceinline__ float shifted(float s, float scale, int lag)
{
    return std::is_same<T, __half>::value ? __fmaf_ru(s, scale, -weight_shift<T>(lag)) : __fmaf_rd(s, scale, -weight_shift<T>(lag));
}

// Key tiles that rows r0 .. r1 of a sequence see: the first one and how many.
struct Span {
    int first, n;
    int lo, hi;       // positions lo .. hi that at least one of the rows sees

    // The tiles of one of so many parts: the first so many have one more.
    __device__ __forceinline__ void part(int i, int parts, int &t0, int &t1) const
    {
        const int each = n / parts, more = n - each * parts;
        t0 = first + i * each + min(i, more);
        t1 = t0 + each + (i < more);
    }
};

template <int TILE>
__device__ __forceinline__ Span span_of(const Attn &a, const Seq &s, int r0, int r1)
{
    const int i0 = a.by_group(r0), i1 = a.by_group(r1);
    Span t;
    t.hi = min(s.pos0 + i1, s.end - 1);
    t.lo = a.window ? max(s.pos0 + i0 - a.window + 1, 0) : 0;
    t.first = t.lo / TILE;
    t.n = t.hi < t.lo ? 0 : t.hi / TILE - t.first + 1;
    return t;
}

// ---------------------------------------------------------------------------------------
// The units of a batch of chunks, counted by a warp: lane j counts sequences j * per ... of the batch.  In a
// sequence the last row tiles come first, which are the longest; of up to 32 sequences the longest of all come first,
// where the CTAs take several units each (4 prompts of 1505 tokens: units of 12 to 1 key tiles; sequence by sequence a CTA
// would have up to 26 tiles, so 14).  Every member is called by whole warps.
// ---------------------------------------------------------------------------------------
struct Unit {
    int b, h, tile, part, parts;
    int slot;                       // of the row tile's first part (parts > 1)
    Seq s;
};

// FEW: up to 32 sequences, one a lane.  (Kernels of their own: a CTA meets the code for the first time, and waits for it;
// 509 tokens at 16384 110 us with both in one, 103 so; 8192 tokens 326 and 321.)
template <int ROWS, int TILE, bool FEW>
struct Plan {
    int per;                        // sequences a lane
    int length;                     // key tiles a part
    int total, split;               // units; rows of row tiles in several parts
    // Before the lane's first sequence: units, slots, rows in several parts.  And, of one sequence a lane, what it is.
    int units, slots, rows;
    Seq s;
    int tiles, parts;
    int top;                        // the last key tile of all, plus 1; 0: units stand sequence by sequence

    // Row tiles of a sequence and the parts of each.
    __device__ __forceinline__ void shape(const Attn &a, const Seq &q, int &t, int &p) const
    {
        const int rows = q.n * a.group;
        t = (rows + ROWS - 1) / ROWS;
        p = t ? max(1, (span_of<TILE>(a, q, (t - 1) * ROWS, rows - 1).n + length - 1) / length) : 0;
    }

    // Up to 32 sequences: the length of a part by trying 32 of them, a lane each, on an estimate of the time of
    // the slowest CTA.  A batch of equal units takes whole rounds of the CTAs; one of unequal units its average and
    // one more unit.
    __device__ __forceinline__ int best_length(const Attn &a, int rows, int first, int last) const
    {
        const int lane = threadIdx.x & 31, mine = (rows + ROWS - 1) / ROWS * a.p.heads;     // row tiles of the lane's sequence
        int most = last, all = mine;
        float work = 0.5f * (float)mine * (float)(first + last);
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
            all += __shfl_xor_sync(0xffffffffu, all, o);
            work += __shfl_xor_sync(0xffffffffu, work, o);
        }
        if (most <= a.least || all <= 0) return max(most, 1);
        // Parts of the longest row tile: what makes 1/8 .. 32/8 rounds of the CTAs; one is always tried.
        int p = lane ? min((int)((float)(lane + 1) * (float)a.ctas / (8.0f * (float)all)), most / a.least) : 1;
        p = max(p, 1);
        const int len = (most + p - 1) / p;
        float count = 0.0f, cut = 0.0f;             // units, and those of row tiles in several parts (exact below 2^24)
        for (int b = 0; b < a.p.seqs; ++b) {
            const int t = __shfl_sync(0xffffffffu, mine, b), n = __shfl_sync(0xffffffffu, last, b);
            const int k = max((n + len - 1) / len, 1);
            const float c = (float)t * (float)k;
            count += c;
            if (k > 1) cut += c;
        }
        const float g = (float)a.ctas, longest = (float)len + a.unit_cost;
        float cost = min(ceilf(count / g) * longest, (work + a.unit_cost * count) / g + longest);
        if (cut > 0.0f) cost += a.unit_cost;
        if (cut > (float)a.slots) cost = INFINITY;
        int best = len;
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const float c = __shfl_xor_sync(0xffffffffu, cost, o);
            const int l = __shfl_xor_sync(0xffffffffu, best, o);
            if (c < cost || (c == cost && l > best)) {
                cost = c;
                best = l;
            }
        }
        return best;
    }

    __device__ __forceinline__ void make(const Attn &a)
    {
        const int lane = threadIdx.x & 31;
        per = (a.p.seqs + 31) / 32;
        const int b0 = min(lane * per, a.p.seqs), b1 = min(b0 + per, a.p.seqs);
        int v[3] = {0, 0, 0};
        if constexpr (FEW) {
            s = Seq{0, 0, 0, 0};
            int n = 0, first = 0, last = 0;
            if (lane < a.p.seqs) {
                s = seq_of(a.p, lane);
                n = s.n * a.group;
                if (n) {
                    first = span_of<TILE>(a, s, 0, min(n, ROWS) - 1).n;
                    last = span_of<TILE>(a, s, (n - 1) / ROWS * ROWS, n - 1).n;
                }
            }
            length = best_length(a, n, first, last);
            tiles = (n + ROWS - 1) / ROWS;
            parts = tiles ? max(1, (last + length - 1) / length) : 0;
            v[0] = tiles * parts * a.p.heads;
            v[1] = parts > 1 ? v[0] : 0;
            v[2] = parts > 1 ? n * a.p.heads : 0;           // (few: the workspace has room for their row tiles)
        } else {
            // Parts of equal length, as many as the workspace has room for: a row tile of p > 1 parts has more than
            // (p - 1) * length >= p * length / 2 key tiles, so there are fewer than twice work / length of them.
            long long w = 0;
#pragma unroll 4
            for (int b = b0; b < b1; ++b) {
                const Seq q = seq_of(a.p, b);
                const int n = q.n * a.group;
                if (n) w += (long long)((n + ROWS - 1) / ROWS) * span_of<TILE>(a, q, (n - 1) / ROWS * ROWS, n - 1).n;
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
            w = (2 * w * a.p.heads + a.slots - 1) / a.slots;
            length = (int)min(max(w, (long long)a.least), (long long)INT_MAX / 2);
#pragma unroll 4
            for (int b = b0; b < b1; ++b) {
                int t, p;
                const Seq q = seq_of(a.p, b);
                shape(a, q, t, p);
                v[0] = min(v[0] + t * a.p.heads * p, (1 << 26) - 1);     // (more only where starts do not ascend)
                if (p > 1) {
                    v[1] += t * a.p.heads * p;
                    v[2] += q.n * a.group * a.p.heads;
                }
            }
        }
        int sum[3];
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            sum[i] = v[i];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, sum[i], o);
                if (lane >= o) sum[i] += u;
            }
        }
        units = sum[0] - v[0];
        slots = sum[1] - v[1];
        rows = sum[2] - v[2];
        total = __shfl_sync(0xffffffffu, sum[0], 31);
        top = 0;
        if (FEW && a.p.seqs > 1 && total > a.ctas) top = __reduce_max_sync(0xffffffffu, tiles ? (s.pos0 + s.n - 1) / TILE + 1 : 1);
        split = __shfl_sync(0xffffffffu, sum[2], 31);
    }

    // The sequence of unit (or, of row tiles in several parts, row) u, and what is left of u in it.
    template <bool JOIN>
    __device__ __forceinline__ Unit sequence(const Attn &a, int u, int &left, int &t) const
    {
        const int before = JOIN ? rows : units;
        const int lo = __popc(__ballot_sync(0xffffffffu, before <= u)) - 1;       // the last lane that starts at or before u
        Unit x;
        left = u - __shfl_sync(0xffffffffu, before, lo);
        x.slot = __shfl_sync(0xffffffffu, slots, lo);
        x.b = lo;
        if constexpr (FEW) {
            x.s.row0 = __shfl_sync(0xffffffffu, s.row0, lo);
            x.s.n = __shfl_sync(0xffffffffu, s.n, lo);
            x.s.pos0 = __shfl_sync(0xffffffffu, s.pos0, lo);
            x.s.end = __shfl_sync(0xffffffffu, s.end, lo);
            t = __shfl_sync(0xffffffffu, tiles, lo);
            x.parts = __shfl_sync(0xffffffffu, parts, lo);
            return x;
        }
        // 32 of the lane's sequences at a time (ends: u < total).
        const int end = min(lo * per + per, a.p.seqs);
        for (int b0 = lo * per;; b0 += 32) {
            const int lane = threadIdx.x & 31;
            Seq q{0, 0, 0, 0};
            int n = 0, p = 0;
            if (b0 + lane < end) {
                q = seq_of(a.p, b0 + lane);
                shape(a, q, n, p);
            }
            const int k = n * a.p.heads * p, mine = !JOIN ? k : p > 1 ? q.n * a.group * a.p.heads : 0, cut = p > 1 ? k : 0;
            int sum = mine, sum_cut = cut;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, sum, o), w = __shfl_up_sync(0xffffffffu, sum_cut, o);
                if (lane >= o) {
                    sum += v;
                    sum_cut += w;
                }
            }
            const int all = __shfl_sync(0xffffffffu, sum, 31);
            if (left >= all && b0 + 32 < end) {
                left -= all;
                x.slot += __shfl_sync(0xffffffffu, sum_cut, 31);
                continue;
            }
            const int at = min(__popc(__ballot_sync(0xffffffffu, sum <= left)), 31);        // the first that reaches beyond it
            left -= __shfl_sync(0xffffffffu, sum - mine, at);
            x.slot += __shfl_sync(0xffffffffu, sum_cut - cut, at);
            x.b = b0 + at;
            x.s.row0 = __shfl_sync(0xffffffffu, q.row0, at);
            x.s.n = __shfl_sync(0xffffffffu, q.n, at);
            x.s.pos0 = __shfl_sync(0xffffffffu, q.pos0, at);
            x.s.end = __shfl_sync(0xffffffffu, q.end, at);
            t = __shfl_sync(0xffffffffu, n, at);
            x.parts = __shfl_sync(0xffffffffu, p, at);
            break;
        }
        return x;
    }
    // (top > 0) How many row tiles of the lane's sequence have their last row at key tile l - 1 or a later one.
    __device__ __forceinline__ int at_least(const Attn &a, int l) const
    {
        const long long x = l ? (long long)(l - 1) * TILE - s.pos0 : 0;      // a row tile has a row of token x or a later one
        return x <= 0 ? tiles : x >= s.n ? 0 : tiles - (int)x * a.group / ROWS;
    }
    // Unit u of them by where their last rows are, latest first.
    __device__ __forceinline__ Unit find_by_length(const Attn &a, int u) const
    {
        const int each = parts * a.p.heads;           // units of a row tile of the lane's sequence
        int lo = 0, hi = top + 1, later = 0;          // more than u units at lo or later, no more than u at hi: `later`
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1, n = __reduce_add_sync(0xffffffffu, at_least(a, mid) * each);
            if (n > u) {
                lo = mid;
            } else {
                hi = mid;
                later = n;
            }
        }
        const int behind = at_least(a, hi), mine = (at_least(a, lo) - behind) * each;
        int sum = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, sum, o);
            if ((threadIdx.x & 31) >= o) sum += v;
        }
        Unit x;
        x.b = __popc(__ballot_sync(0xffffffffu, sum <= u - later));          // the first lane that reaches beyond u
        const int left = u - later - __shfl_sync(0xffffffffu, sum - mine, x.b);
        x.s.row0 = __shfl_sync(0xffffffffu, s.row0, x.b);
        x.s.n = __shfl_sync(0xffffffffu, s.n, x.b);
        x.s.pos0 = __shfl_sync(0xffffffffu, s.pos0, x.b);
        x.s.end = __shfl_sync(0xffffffffu, s.end, x.b);
        x.parts = __shfl_sync(0xffffffffu, parts, x.b);
        const int item = left / x.parts;
        x.part = left - item * x.parts;
        const int k = a.by_heads(item) + __shfl_sync(0xffffffffu, behind, x.b);      // row tiles of the sequence behind it
        x.tile = __shfl_sync(0xffffffffu, tiles, x.b) - 1 - k;
        x.h = item - a.by_heads(item) * a.p.heads;
        x.slot = __shfl_sync(0xffffffffu, slots, x.b) + (k * a.p.heads + x.h) * x.parts;
        return x;
    }

    __device__ __forceinline__ Unit find(const Attn &a, int u) const
    {
        if constexpr (FEW)
            if (top > 0) return find_by_length(a, u);
        int left, t;
        Unit x = sequence<false>(a, u, left, t);
        const int item = x.parts == 1 ? left : left / x.parts;
        x.part = left - item * x.parts;
        x.tile = t - 1 - a.by_heads(item);
        x.h = item - a.by_heads(item) * a.p.heads;
        x.slot += item * x.parts;
        return x;
    }
    // Where row i of those in several parts stands: its sequence, head and row of these; tile is how many row tiles there
    // are, slot that of the sequence's first part.
    __device__ __forceinline__ Unit find_row(const Attn &a, int i, int &row) const
    {
        int left, t;
        Unit x = sequence<true>(a, i, left, t);
        x.tile = t;
        x.part = 0;
        x.h = left / (x.s.n * a.group);
        row = left - x.h * x.s.n * a.group;
        return x;
    }
};

// ---------------------------------------------------------------------------------------
// Output
// ---------------------------------------------------------------------------------------
// Four consecutive values of `type`, 16-byte aligned as f32 and 8-byte aligned otherwise.
__device__ __forceinline__ void store4(void *p, int type, float4 v)
{
    if (type == Q8ACT_F32) {
        *static_cast<float4 *>(p) = v;
    } else if (type == Q8ACT_F16) {
        const __half2 a = __floats2half2_rn(v.x, v.y), b = __floats2half2_rn(v.z, v.w);
        *static_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    } else {
        const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
        *static_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    }
}

__device__ __forceinline__ int out_size(int type) { return type == Q8ACT_F32 ? 4 : 2; }

// ---------------------------------------------------------------------------------------
// Non-finite values in places that only some rows of a tile see.  The tensor cores multiply every
// value of a tile by every row's weight, and 0 times infinity or NaN is NaN: a row would be spoilt by a
// value that its mask hides from it.  So values that no row of the unit sees are cleared, and so are non-finite ones of
// positions that only some rows see; what the latter give the rows that see them is added here:
//   acc[j] += exp2(score - mx) v[position][col(j)]  over the non-finite v of positions k0 .. k1
// These positions are no more than the unit's tokens, at either end of what it sees.  (A position added twice
// changes nothing: what it adds is not finite.)
// ---------------------------------------------------------------------------------------
template <typename T, int D, int N, typename Col>
__device__ __noinline__ void add_non_finite(const Attn &a, int b, int h, const T *q, int k0, int k1, float mx, Col col,
                                            float (&acc)[N])
{
    const T *kc = static_cast<const T *>(a.kc), *vc = static_cast<const T *>(a.vc);
    const int64_t head_stride = (int64_t)D << a.p.page_shift;
    for (int k = k0; k <= k1; ++k) {
        const int64_t page = page_of(a.p, b, k >> a.p.page_shift);
        if (page < 0) continue;
        const int64_t at = page * a.p.page_stride + h * head_stride + (int64_t)(k & ((1 << a.p.page_shift) - 1)) * D;
        bool some = false;
        for (int j = 0; j < N; ++j) some |= !isfinite(to_f32(vc[at + col(j)]));
        if (!some) continue;
        float s = 0.0f;
        for (int i = 0; i < D; ++i) s = fmaf(to_f32(q[i]), to_f32(kc[at + i]), s);
        const float p = attn_ex2(fmaf(s, a.scale, -mx));
        for (int j = 0; j < N; ++j) {
            const float v = to_f32(vc[at + col(j)]);
            if (!isfinite(v)) acc[j] = fmaf(p, v, acc[j]);
        }
    }
}

// ---------------------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------------------
inline size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// Workspace for so many partial results of row tiles.
inline size_t attention_space(int slots, int rows, int dim)
{
    return up256((size_t)slots * rows * sizeof(float2)) + (size_t)slots * rows * dim * sizeof(float);
}
inline void attention_place(Attn &a, void *ws, int slots, int rows)
{
    a.slots = slots;
    a.ml = static_cast<float2 *>(ws);
    a.part = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + up256((size_t)slots * rows * sizeof(float2)));
}

inline CUtensorMapDataType attention_type(const q8act_paged_kv &kv)
{
    return kv.type == Q8ACT_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
}

// Tensor maps of the cache, boxes of 64 values x `rows` positions of a page.
inline bool attention_maps(const q8act_paged_kv &kv, int rows, CUtensorMap *tk, CUtensorMap *tv)
{
    const CUtensorMapDataType dt = attention_type(kv);
    const uint64_t dims[4] = {(uint64_t)kv.dim, (uint64_t)kv.page_size, (uint64_t)kv.heads, (uint64_t)kv.pages};
    const uint64_t strides[3] = {(uint64_t)kv.dim * 2, (uint64_t)kv.dim * 2 * kv.page_size, (uint64_t)kv.page_stride * 2};
    const uint32_t box[4] = {64, (uint32_t)(kv.page_size < rows ? kv.page_size : rows), 1, 1};
    return encode_tiled(tk, dt, kv.k, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) &&
           encode_tiled(tv, dt, kv.v, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// The kernel for chunks (attention_tc.cu): its workspace, its launch (a: all but how units are cut), and the joining
// kernel behind either.
constexpr int CHUNK_ROWS = 256, CHUNK_TILE = 128;
size_t attention_chunk_space(int dim);
cudaError_t launch_attention_chunk(const DeviceInfo &dev, const q8act_paged_kv &kv, Attn a, void *ws, cudaStream_t stream);
cudaError_t launch_attention_chunk_join(const DeviceInfo &dev, const Attn &a, int dim, cudaStream_t stream);

}  // namespace q8
