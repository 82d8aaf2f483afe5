// attention.cuh -- what the attention kernels share: how a batch is cut into units of work, masks,
// the exact way round non-finite values, partial results and output.
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

// A row tile in several parts, as the joining kernel needs it: the slot of its first part, its place.
struct Item {
    int slot, parts, row0, first, h, rows, unused[2];    // first: its first row among the sequence's, which start at row0
};

// Division of 0 .. 2^31 - 1 by a number that the launch fixes.
struct Divide {
    uint32_t by, factor, shift;
    Divide(uint32_t d = 1) : by(d)
    {
        shift = 0;
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
    int target, least;           // parts to aim at, and the fewest key tiles that a part is worth
    float scale;                 // of scores, times log2 e
    // partial results of row tiles in several parts (attention_workspace)
    int32_t *count;              // of such row tiles
    Item *items;
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
// The units of a batch, counted by the CTA's first NT threads: thread j counts sequences j * per ... of the
// batch.  The last row tiles come first, which are the longest.
// ---------------------------------------------------------------------------------------
template <int NT>
struct PlanSmem {
    int units[NT + 1], slots[NT + 1], items[NT + 1];    // before thread j's sequences
    long long work[NT / 32];
    int sums[3][NT / 32];
};

struct Unit {
    int b, h, tile, part, parts;
    int slot, item;                 // of the row tile's first part (parts > 1)
    Seq s;
};

template <int ROWS, int TILE, int NT>
struct Plan {
    int per;       // sequences a thread
    int length;    // key tiles a part
    int total;     // units

    // Row tiles of a sequence and the parts of each.
    __device__ __forceinline__ void shape(const Attn &a, const Seq &s, int &tiles, int &parts) const
    {
        const int rows = s.n * a.group;
        tiles = (rows + ROWS - 1) / ROWS;
        parts = tiles ? max(1, (span_of<TILE>(a, s, (tiles - 1) * ROWS, rows - 1).n + length - 1) / length) : 0;
    }

    // Called by all threads of the CTA.
    __device__ __forceinline__ void make(const Attn &a, PlanSmem<NT> &sm)
    {
        const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
        const bool counts = t < NT;
        per = (a.p.seqs + NT - 1) / NT;
        const int b0 = counts ? min(t * per, a.p.seqs) : 0, b1 = counts ? min(b0 + per, a.p.seqs) : 0;
        long long w = 0;
        for (int b = b0; b < b1; ++b) {
            const Seq s = seq_of(a.p, b);
            const int rows = s.n * a.group;
            if (rows) w += (long long)((rows + ROWS - 1) / ROWS) *
                           span_of<TILE>(a, s, (rows - 1) / ROWS * ROWS, rows - 1).n;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
        if (counts && lane == 0) sm.work[warp] = w;
        __syncthreads();
        w = 0;
#pragma unroll
        for (int i = 0; i < NT / 32; ++i) w += sm.work[i];
        w = (w * a.p.heads + a.target - 1) / a.target;
        length = (int)min(max(w, (long long)a.least), (long long)INT_MAX / 2);

        int v[3] = {0, 0, 0};
        for (int b = b0; b < b1; ++b) {
            const Seq s = seq_of(a.p, b);
            int tiles, parts;
            shape(a, s, tiles, parts);
            tiles *= a.p.heads;
            v[0] += tiles * parts;
            if (parts > 1) {
                v[1] += tiles * parts;
                v[2] += tiles;
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
            if (counts && lane == 31) sm.sums[i][warp] = sum[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 3; ++i) {
#pragma unroll
            for (int j = 0; j < NT / 32; ++j)
                if (j < warp) sum[i] += sm.sums[i][j];
        }
        if (counts) {
            sm.units[t] = sum[0] - v[0];
            sm.slots[t] = sum[1] - v[1];
            sm.items[t] = sum[2] - v[2];
        }
        if (t == NT - 1) {
            sm.units[NT] = sum[0];
            sm.slots[NT] = sum[1];
            sm.items[NT] = sum[2];
        }
        __syncthreads();
        total = sm.units[NT];
    }

    // Called by whole warps.
    __device__ __forceinline__ Unit find(const Attn &a, const PlanSmem<NT> &sm, int u) const
    {
        int lo = -1;                                // the last thread that starts at or before u
#pragma unroll
        for (int i = 0; i < NT; i += 32) lo += __popc(__ballot_sync(0xffffffffu, sm.units[i + (threadIdx.x & 31)] <= u));
        Unit x;
        int left = u - sm.units[lo], tiles, parts;
        x.slot = sm.slots[lo];
        x.item = sm.items[lo];
        for (x.b = lo * per;; ++x.b) {              // ends: u < total
            x.s = seq_of(a.p, x.b);
            shape(a, x.s, tiles, parts);
            const int n = tiles * parts * a.p.heads;
            if (left < n || x.b + 1 >= a.p.seqs) break;
            left -= n;
            if (parts > 1) {
                x.slot += n;
                x.item += tiles * a.p.heads;
            }
        }
        x.parts = parts;
        x.part = left % parts;
        const int it = left / parts;
        x.tile = tiles - 1 - a.by_heads(it);
        x.h = it - a.by_heads(it) * a.p.heads;
        x.slot += it * parts;
        x.item += it;
        return x;
    }
};

// ---------------------------------------------------------------------------------------
// Output
// ---------------------------------------------------------------------------------------
// N consecutive values of `type` (4, 8 or 16 of them, 16-byte aligned where they fill 16 bytes).
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
// value that its mask hides from it.  Values that no row of the unit sees are cleared; where some rows
// see a non-finite one, the unit's sums of weighted values are taken again here, value by value and
// only over what the row sees.  Slow, and reached by such inputs only.
// acc[j] = sum over positions k0 .. k1 of exp2(score - mx) v[position][col(j)]
// ---------------------------------------------------------------------------------------
template <typename T, int D, int N, typename Col>
__device__ __noinline__ void exact_values(const Attn &a, int b, int h, const T *q, int k0, int k1, float mx, Col col,
                                          float (&acc)[N])
{
    const T *kc = static_cast<const T *>(a.kc), *vc = static_cast<const T *>(a.vc);
    const int64_t head_stride = (int64_t)D << a.p.page_shift;
    for (int j = 0; j < N; ++j) acc[j] = 0.0f;
    for (int k = k0; k <= k1; ++k) {
        const int64_t page = page_of(a.p, b, k >> a.p.page_shift);
        if (page < 0) continue;
        const int64_t at = page * a.p.page_stride + h * head_stride + (int64_t)(k & ((1 << a.p.page_shift) - 1)) * D;
        float s = 0.0f;
        for (int i = 0; i < D; ++i) s = fmaf(to_f32(q[i]), to_f32(kc[at + i]), s);
        const float p = attn_ex2(fmaf(s, a.scale, -mx));
        for (int j = 0; j < N; ++j) acc[j] = fmaf(p, to_f32(vc[at + col(j)]), acc[j]);
    }
}

// A row's maximum and sum over the same positions.
template <typename T, int D>
__device__ __noinline__ float2 exact_statistics(const Attn &a, int b, int h, const T *q, int k0, int k1)
{
    const T *kc = static_cast<const T *>(a.kc);
    const int64_t head_stride = (int64_t)D << a.p.page_shift;
    float mx = -INFINITY, sum = 0.0f;
    for (int k = k0; k <= k1; ++k) {
        const int64_t page = page_of(a.p, b, k >> a.p.page_shift);
        if (page < 0) continue;
        const int64_t at = page * a.p.page_stride + h * head_stride + (int64_t)(k & ((1 << a.p.page_shift) - 1)) * D;
        float s = 0.0f;
        for (int i = 0; i < D; ++i) s = fmaf(to_f32(q[i]), to_f32(kc[at + i]), s);
        const float m = fmaxf(mx, s * a.scale), base = m == -INFINITY ? 0.0f : m;
        sum = sum * attn_ex2(mx - base) + attn_ex2(fmaf(s, a.scale, -base));
        mx = m;
    }
    return make_float2(mx, sum);
}

// ---------------------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------------------
inline size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// Workspace for `target` parts of `rows` rows: a row tile of p > 1 parts has more than
// (p - 1) * length >= p * length / 2 key tiles, so there are fewer slots than twice the target, and half as
// many items.
inline size_t attention_space(int target, int rows, int dim)
{
    const size_t slots = 2 * (size_t)target;
    return 256 + up256(slots / 2 * sizeof(Item)) + up256(slots * rows * sizeof(float2)) + slots * rows * (size_t)dim * sizeof(float);
}
inline void attention_place(Attn &a, void *ws, int target, int rows)
{
    const size_t slots = 2 * (size_t)target;
    uint8_t *p = static_cast<uint8_t *>(ws);
    a.target = target;
    a.count = reinterpret_cast<int32_t *>(p);
    a.items = reinterpret_cast<Item *>(p + 256);
    a.ml = reinterpret_cast<float2 *>(p + 256 + up256(slots / 2 * sizeof(Item)));
    a.part = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(a.ml) + up256(slots * rows * sizeof(float2)));
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

// The kernel for chunks (attention_tc.cu): its workspace, its launch (a: all but the workspace's places), and
// the joining kernel behind either.
constexpr int CHUNK_ROWS = 256;
size_t attention_chunk_space(int dim);
cudaError_t launch_attention_chunk(const DeviceInfo &dev, const q8act_paged_kv &kv, Attn a, void *ws, cudaStream_t stream);
cudaError_t launch_attention_join(const DeviceInfo &dev, const Attn &a, int dim, int rows, cudaStream_t stream);

}  // namespace q8
