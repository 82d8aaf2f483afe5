// attention_tc.cu -- attention of chunks of new tokens over a paged cache on the tensor cores (tcgen05).
//   S = Q K^T,  P = e^(scale S - mx),  O = P V,  out = O / sum P
//
// A CTA holds two tiles of 128 rows (query heads of a group x tokens) and walks over tiles of 128
// positions.  S and O are accumulators in tensor memory; P, rounded to the cache's type, is the second product's
// first operand from there, so only Q, K and V go through shared memory.  With 128 values a head the 512 columns
// are full with two S and two O, so P takes the place of S: while the four warps of one row tile turn S into P,
// the tensor cores work for the other tile.  With 64 values P has columns of its own, and the next S is computed
// while its row tile's warps are still at work on this one.
//   warps 0-3, 4-7  a row tile each: a thread a row, so maxima and sums need no exchange
//   warp 8          issues the MMAs, K' the next tile's keys: P0 V, Q0 K', P1 V, Q1 K', or (P apart) Q0 K', P1 V of
//                   the tile before, Q1 K', P0 V
//   warp 9          brings pages of keys and values to shared memory (TMA, 128-byte swizzled)
//   warp 10         in tiles of values that some row does not see as a whole clears those that no row sees, and
//                   infinities and NaN among those that only some see (attention.cuh)
//   warp 11         works out the CTA's next units for the others, and brings their queries
// O is rescaled only when a row's maximum has risen by more than 2^8 since the last time: until then P is
// at most 2^8 (times a power of two, weight_shift) and nothing is lost (f32 sums, the type's relative precision).
//
// Bound by the tensor cores and by what they wait for.  128 values a head: 8192 tokens of 32 + 8 heads bf16 319 us
// (1.72 PFLOP/s, 0.91 of cuBLAS's bf16 burst rate), the tensor pipe 76 % busy; a step of both row tiles is 2048 tensor
// cycles and takes about 2450, the chain of one row tile: S 230 cycles after its MMAs, maximum 490, weights 1000 (P in two
// parts, the products of the first under way), products and next S 800.  64 values: 64 + 8 heads, 8000 tokens, window 1024 f16
// 168 us, where the exponentials bound: 2 x 128 a thread of the four schedulers' 8 a cycle are 1024 cycles a step, with the
// rest of the softmax 1900; ten tiles a unit, of which three are masked, leave 3400 cycles between units beside them.
// What was tried without gain: a thread half a row (640 threads: registers spill), S twice through registers
// (the loads' latency), P in four parts, a warp of its own for the output (512 threads leave 128 registers), an MMA
// warp a row tile (they fall into step: 457 us), both halves on the same rows with every other tile (35 rows, 6000
// positions: 31 -> 42 us), equal stretches as for few tokens (a cut costs two f32 outputs, a change of units and the
// join: 509 tokens at 16384 110 -> 125 us), the next S of a row tile alone in the other's place (16 x 5 tokens at 6000, one row
// tile each, 24.1 -> 23.7 us: 1.2 us a key tile of 152 CTAs is the copy rate).
#include <algorithm>

#include "attention.cuh"

namespace q8 {
namespace {

constexpr int TILE = CHUNK_TILE;         // positions a step
constexpr int QROWS = 128;               // rows of a row tile
constexpr int ROWS = CHUNK_ROWS;         // of a unit: two row tiles
constexpr int THREADS = 384;
constexpr int SOFTMAX_REGS = 208, OTHER_REGS = 88;      // 256 x 208 + 128 x 88 = 384 x 168, the launch's registers
constexpr int PARTS = 2;                 // of a tile's weights, handed to the MMAs one by one
constexpr float NEG = -INFINITY;
constexpr int SLACK = 8;
constexpr int OUT_BYTES = 32 * 128;

template <int D>
struct Cfg {
    static constexpr int Q_BYTES = QROWS * D * 2;              // a row tile's queries
    static constexpr int STAGE_BYTES = TILE * D * 2;           // a tile of keys or of values
    static constexpr int STAGES = 128 * 1024 / STAGE_BYTES;
    static constexpr int HALVES = D / 64;                      // columns of 128 bytes
    static constexpr int HALF_BYTES = TILE * 128;
    static constexpr int OFF_OUT = 2 * Q_BYTES + STAGES * STAGE_BYTES;      // a softmax warp's 32 rows x 128 bytes on their way out
    static constexpr int OFF_SHARED = OFF_OUT + 8 * OUT_BYTES;
    // Tensor memory: S0 S1 O0 O1, and P0 P1 where there is room for them.  Where there is not, P takes the place of S.
    static constexpr bool OWN_P = 2 * (TILE + D + TILE / 2) <= 512;
    static constexpr uint32_t COL_S = 0, COL_O = 2 * TILE, COL_P = OWN_P ? COL_O + 2 * D : COL_S, P_STRIDE = OWN_P ? TILE / 2 : TILE;
    // Instruction descriptor, kind::f16: D f32 (bits 4-5), types of A and B (7-9, 10-12), B's major (16; 1: its
    // rows are K), N >> 3 (17-22), M >> 4 (24-28).
    static constexpr uint32_t IDESC_QK = (1u << 4) | ((uint32_t)(TILE >> 3) << 17) | ((uint32_t)(QROWS >> 4) << 24);
    static constexpr uint32_t IDESC_PV = (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | ((uint32_t)(QROWS >> 4) << 24);
    static constexpr uint32_t IDESC_BF16 = (1u << 7) | (1u << 10);
};

// A unit, as its roles need it: tiles [t0, t1) (t0 < 0: no more units), those that row tile q sees, [a[q], b[q]).
struct Record {
    int t0, t1, a[2], b[2];
    int lo, hi;              // positions that at least one row sees
    int first, last;         // positions of the first and the last row
    int row0, rows, r0, h;   // the sequence's first token, its rows, the unit's first one; head of keys and values
    int pos0, end, seq;      // position of the sequence's first row, positions in the cache, sequence
    int slot;                // of the unit in the partial results, or -1

    // Whether some row does not see some of a tile.
    __device__ __forceinline__ bool masked(const Attn &at, int t) const
    {
        return t * TILE < lo || t * TILE + TILE - 1 > min(first, hi) || (at.window && t * TILE <= last - at.window);
    }
};
constexpr int RECORDS = 4;                         // units known in advance, at most
constexpr int READERS = 8 + 1 + 1 + 1;             // warps that read them: all but warp 11

struct Shared {
    uint64_t full[8], empty[8];                      // stages
    // Tile n of the CTA, in barrier n % 8: its values, and the next tile's keys, are there.  The stages hold four tiles
    // at most, so five barriers would do.
    uint64_t ready[8];
    uint64_t s_full[2], p_full[2][PARTS], q_full[2], q_empty[2], o_full[2], drained;
    uint64_t s_empty[2], p_empty[2];                 // (P apart) S is in registers, P V is done
    uint64_t unit_full[RECORDS], unit_empty[RECORDS];
    Record units[RECORDS];
    uint32_t pages[8];                               // tile n of the CTA in word n % 8: its 16-position blocks whose page exists
    uint32_t tmem;
    // Unit n of the CTA, counting those with positions, has had a non-finite value cleared that some rows see: n + 1 in word
    // n % 16.  Warp 10 is ahead of the softmax by the stages' tiles at most, 4 and one.
    uint32_t spoilt[16];
    int abort_flag;
};

// V's tile [position][64 values of a half], 128-byte swizzled, as the operand whose rows are K: 64-value
// blocks HALF_BYTES apart (leading dimension), groups of 8 positions 1024 bytes apart (stride).
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t saddr, uint32_t block_bytes)
{
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(block_bytes >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}

// 32 columns of the warp's 32 lanes, a lane a thread; the registers are valid after wait_ld.
__device__ __forceinline__ void ld32(uint32_t taddr, float *r)
{
    uint32_t *u = reinterpret_cast<uint32_t *>(r);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
          "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]), "=r"(u[16]),
          "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]),
          "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
        : "r"(taddr));
}
template <int N>
__device__ __forceinline__ void wait_ld(float *r)
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+f"(r[i]));
}
__device__ __forceinline__ void st32(uint32_t taddr, const uint32_t *u)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
        ::"r"(taddr), "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]),
          "r"(u[9]), "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15]), "r"(u[16]), "r"(u[17]),
          "r"(u[18]), "r"(u[19]), "r"(u[20]), "r"(u[21]), "r"(u[22]), "r"(u[23]), "r"(u[24]), "r"(u[25]), "r"(u[26]),
          "r"(u[27]), "r"(u[28]), "r"(u[29]), "r"(u[30]), "r"(u[31])
        : "memory");
}
// The lowest n bits of a word, none or all where n is out of range.
__device__ __forceinline__ uint32_t bits_below(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1; }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 16 bytes from global to shared memory, of which the first `bytes` are read and the others zeros.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint32_t bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// 128 bytes of each lane's row, through the warp's part of shared memory: a store then writes four rows' whole
// lines instead of 16 bytes of 32.  dst: where the lane's row goes (null: nowhere).
__device__ __forceinline__ void store_rows(uint8_t *out, const uint4 (&v)[8], uint8_t *dst, int off)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 0; k < 8; ++k) *reinterpret_cast<uint4 *>(out + lane * 128 + ((k ^ (lane & 7)) << 4)) = v[k];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = 4 * i + (lane >> 3), k = lane & 7;
        uint8_t *p = reinterpret_cast<uint8_t *>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(dst), row));
        if (p) *reinterpret_cast<uint4 *>(p + off + k * 16) = *reinterpret_cast<const uint4 *>(out + row * 128 + ((k ^ (row & 7)) << 4));
    }
    __syncwarp();
}

// A whole warp's wait for one barrier; one look where it is over.
__device__ __forceinline__ bool arrived(uint64_t *bar, uint32_t parity, int *status, volatile int *abort_flag)
{
    return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) ||
           __all_sync(0xffffffffu, wait_or_abort(bar, parity, status, abort_flag));
}

// What a row's weights 2^(s scale - mx) are relative to, and the scale.
//
// The exponent is one fma, exact but for its result's rounding, so for the largest score it is the shift and what the product in mx
// has been rounded by: less than 8 up to FAR.  Beyond, scores themselves are 4 and more apart, and that would leave no weight at
// all: a power of two takes the scale's place there, whose products are exact.  So equal scores have equal weights, whatever their
// size.  (Parts of a row on either side of FAR: the larger score's has all the weight.)  A rounded product and a subtraction, as in
// attention.cu, are twice the instructions on the 128 scores of a thread.
constexpr float FAR = 0x1p26f;

template <typename T>
struct Reference {
    float mx = NEG, scale;

    __device__ __forceinline__ explicit Reference(const Attn &a) : scale(a.scale) {}
    __device__ __forceinline__ float base() const { return mx == NEG ? 0.0f : mx; }
    // mx if the largest score were s.
    __device__ __forceinline__ float with(float s) const { return fmaxf(mx, shifted<T>(s, scale, SLACK)); }
    // The largest score is s now, m = with(s): what the sums so far are to be multiplied by.  (mx may be -inf: they are zeros.)
    __device__ __forceinline__ float rise(const Attn &a, float s, float m)
    {
        if (m > mx) {
            m = shifted<T>(s, a.scale, SLACK);
            const bool far = fabsf(m) > FAR;
            scale = far ? a.far_scale : a.scale;
            if (far) m = shifted<T>(s, a.far_scale, SLACK);
        }
        const float f = attn_ex2(mx - (m == NEG ? 0.0f : m));
        mx = m;
        return f;
    }
};

// The unit of this CTA's round: rounds run forwards and backwards in turn, since earlier units are longer.
__device__ __forceinline__ int64_t unit_of(int round)
{
    const int c = blockIdx.x, g = gridDim.x;
    return (int64_t)round * g + (round & 1 ? g - 1 - c : c);
}

// What cleared non-finite values give columns c0 .. c0 + 63 of a row (attention.cuh).
template <typename T, int D>
__device__ __noinline__ void cleared_part(const Attn &a, const Record &x, int row, int c0, float base, float (&o)[64])
{
    const int r = x.r0 + row, tok = a.by_group(r), pos = x.pos0 + tok;
    const int k0 = max(a.window ? pos - a.window + 1 : 0, x.t0 * TILE), k1 = min(min(pos, x.end - 1), x.t1 * TILE - 1);
    const T *q = static_cast<const T *>(a.q) + (x.row0 + tok) * a.ldq + (x.h * a.group + r - tok * a.group) * D;
    auto col = [&](int j) { return c0 + j; };
    for (int j = 0; j < 64; ++j) o[j] = 0.0f;
    if (a.window) add_non_finite<T, D>(a, x.seq, x.h, q, k0, min(k1, x.last - a.window), base, col, o);
    add_non_finite<T, D>(a, x.seq, x.h, q, max(k0, min(x.first, x.hi) + 1), k1, base, col, o);
}

// Rows r0 .. r1 - 1 of a tile of values, by a warp: cleared outside lo .. hi; whether one inside holds an infinity
// or NaN (in this lane's part).
template <typename T, int D>
__device__ __forceinline__ bool fix_rows(uint8_t *tile, int r0, int r1, int lo, int hi)
{
    using T2 = std::conditional_t<std::is_same<T, __half>::value, __half2, __nv_bfloat162>;
    constexpr int VECS = D / 8, AT_ONCE = 32 / VECS;           // 16-byte vectors of a row, rows a round of lanes
    const int lane = threadIdx.x & 31, v = lane % VECS;
    uint8_t *p = tile + (v >> 3) * (TILE * 128) + (v & 7) * 16;
    uint32_t top[4] = {0, 0, 0, 0};                              // largest magnitudes, NaN above all
#pragma unroll 4
    for (int r = r0 + lane / VECS; r < r1; r += AT_ONCE) {
        uint4 *w = reinterpret_cast<uint4 *>(p + r * 128);
        if (r < lo || r > hi) {
            *w = make_uint4(0, 0, 0, 0);
        } else {
            const uint4 u = *w;
            const uint32_t us[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const T2 m = __hmax2_nan(*reinterpret_cast<const T2 *>(&top[i]), __habs2(*reinterpret_cast<const T2 *>(&us[i])));
                top[i] = *reinterpret_cast<const uint32_t *>(&m);
            }
        }
    }
    constexpr uint32_t E = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
    bool found = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) found |= (top[i] & E) == E || (top[i] >> 16 & E) == E;
    return found;
}

// Infinities and NaN cleared in rows lo .. hi of a tile but from .. to - 1.
template <typename T, int D>
__device__ __forceinline__ void clear_non_finite(uint8_t *tile, int lo, int hi, int from, int to)
{
    constexpr uint32_t E = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
#pragma unroll 1
    for (int i = threadIdx.x & 31; i < TILE * D / 2; i += 32) {           // 4-byte words, a half of the columns after the other
        const int r = i / 32 % TILE;
        if (r < lo || r > hi || (r >= from && r < to)) continue;
        uint32_t &w = reinterpret_cast<uint32_t *>(tile)[i];
        w &= ((w & E) == E ? 0xffff0000u : ~0u) & ((w >> 16 & E) == E ? 0x0000ffffu : ~0u);
    }
}

// FEW: up to 32 sequences (Plan).  BOXES: a row tile holds whole tokens, so its queries come as one TMA box; otherwise they are
// gathered row by row.  Kernels of their own, since less code is faster by itself here (64 + 8 heads x 64, window 1024 of
// 8000: 176 us with both ways of queries in one, 168 so).
template <typename T, int D, bool FEW, bool BOXES>
__global__ void __launch_bounds__(THREADS, 1)
    attention_chunk_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                           const __grid_constant__ CUtensorMap tm_q, Attn a)
{
    using C = Cfg<D>;
    constexpr bool BF16 = std::is_same<T, __nv_bfloat16>::value;
    constexpr int STAGES = C::STAGES;
    constexpr uint32_t IDESC_QK = C::IDESC_QK | (BF16 ? C::IDESC_BF16 : 0), IDESC_PV = C::IDESC_PV | (BF16 ? C::IDESC_BF16 : 0);
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *stages = smem + 2 * C::Q_BYTES;
    Shared &sm = *reinterpret_cast<Shared *>(smem + C::OFF_SHARED);
    volatile int *abort_flag = &sm.abort_flag;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) { mbar_init(&sm.full[s], 1); mbar_init(&sm.empty[s], 2); }
        for (int i = 0; i < 8; ++i) mbar_init(&sm.ready[i], 1);
        for (int i = 0; i < RECORDS; ++i) { mbar_init(&sm.unit_full[i], 1); mbar_init(&sm.unit_empty[i], READERS); }
        for (int q = 0; q < 2; ++q) {
            mbar_init(&sm.s_full[q], 1);
            for (int i = 0; i < PARTS; ++i) mbar_init(&sm.p_full[q][i], 4);
            mbar_init(&sm.q_full[q], 1);
            mbar_init(&sm.q_empty[q], 1);
            mbar_init(&sm.o_full[q], 1);
            mbar_init(&sm.s_empty[q], 4);
            mbar_init(&sm.p_empty[q], 1);
        }
        mbar_init(&sm.drained, 1);
        for (int i = 0; i < 16; ++i) sm.spoilt[i] = 0;
        sm.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 8) tc_alloc(&sm.tmem, 512);
    if (warp == 9 && lane == 0) {
        prefetch_tensormap(&tm_k);
        prefetch_tensormap(&tm_v);
        if (BOXES) prefetch_tensormap(&tm_q);
    }
    griddep_wait();
    griddep_launch_dependents();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, sm.tmem, 0);

    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(SOFTMAX_REGS));
        // ------------------------------ softmax ------------------------------
        const int q = warp >> 2, row = (warp & 3) * 32 + lane;         // of the row tile
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;             // the warp's lanes of tensor memory
        const uint32_t col_s = tmem + lanes + C::COL_S + q * TILE, col_o = tmem + lanes + C::COL_O + q * D;
        const uint32_t col_p = tmem + lanes + C::COL_P + q * C::P_STRIDE;
        uint32_t s_phase = 0, o_phase = 0, p_phase = 1, n = 0, tiles = 0;          // n: units with positions so far
        bool ok = true;
        for (int round = 0;; ++round) {
            ok = arrived(&sm.unit_full[round % RECORDS], round / RECORDS & 1, a.status, abort_flag);
            const Record &x = sm.units[round % RECORDS];
            if (!ok || x.t0 < 0) break;
            const int from = x.a[q], end = x.b[q], r = x.r0 + q * QROWS + row;
            const bool live = r < x.rows;
            const int pos = x.pos0 + a.by_group(live ? r : 0);
            const int hi = live ? min(pos, x.end - 1) : INT_MAX - 1, lo = live && a.window ? max(pos - a.window + 1, 0) : 0;
            const uint32_t tiles0 = tiles;               // tile t of the sequence is tile tiles0 + t - t0 of the CTA
            const bool some = end > from;
            tiles += x.t1 - x.t0;
            Reference<T> at(a);
            float sum = 0.0f;
            bool first = true;
            for (int t = from; t < end; ++t) {
                ok = arrived(&sm.s_full[q], s_phase, a.status, abort_flag);
                if (!ok) break;
                s_phase ^= 1;
                tc_fence_after();
                float s[TILE];
#pragma unroll
                for (int i = 0; i < TILE / 32; ++i) ld32(col_s + 32 * i, s + 32 * i);
                const int k0 = t * TILE;
                const uint32_t pages = *const_cast<volatile uint32_t *>(&sm.pages[(tiles0 + t - x.t0) & 7]);
                const bool edge = __any_sync(0xffffffffu, k0 + TILE - 1 > hi || k0 < lo) || pages != 0xff;
                wait_ld<TILE>(s);
                if constexpr (C::OWN_P) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.s_empty[q]);
                }
                if (edge) {
#pragma unroll
                    for (int c = 0; c < TILE / 32; ++c) {
                        const uint32_t seen = bits_below(hi + 1 - k0 - 32 * c) & ~bits_below(lo - k0 - 32 * c) &
                                              ((pages >> (2 * c) & 1 ? 0xffffu : 0u) | (pages >> (2 * c) & 2 ? 0xffff0000u : 0u));
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (!(seen >> j & 1)) s[32 * c + j] = NEG;
                    }
                }
                float m4[8] = {NEG, NEG, NEG, NEG, NEG, NEG, NEG, NEG};
#pragma unroll
                for (int j = 0; j < TILE; j += 16)
#pragma unroll
                    for (int i = 0; i < 8; ++i) m4[i] = fmaxf(fmaxf(m4[i], s[j + 2 * i]), s[j + 2 * i + 1]);
                const float largest = fmaxf(fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])), fmaxf(fmaxf(m4[4], m4[5]), fmaxf(m4[6], m4[7])));
                const float m = at.with(largest);
                if constexpr (C::OWN_P) {           // the last products have taken P, and added to O
                    ok = arrived(&sm.p_empty[q], p_phase, a.status, abort_flag);
                    if (!ok) break;
                    p_phase ^= 1;
                    tc_fence_after();
                }
                if (first) {
                    at.rise(a, largest, m);
                    first = false;
                } else if (__any_sync(0xffffffffu, m > __fadd_rd(at.mx, SLACK))) {
                    const float f = at.rise(a, largest, m);
                    sum *= f;
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) {
                        float o[32];
                        ld32(col_o + 32 * i, o);
                        wait_ld<32>(o);
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] *= f;
                        st32(col_o + 32 * i, reinterpret_cast<const uint32_t *>(o));
                    }
                }
                const float base = at.base();
                const float2 scale2 = make_float2(at.scale, at.scale), base2 = make_float2(-base, -base);
                float2 sum2[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
                for (int c = 0; c < PARTS; ++c) {
                    constexpr int N = TILE / 2 / PARTS;
                    const float *v = s + 2 * N * c;
                    uint32_t p[N];
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        float2 e = __ffma2_rn(make_float2(v[2 * j], v[2 * j + 1]), scale2, base2);
                        e = make_float2(attn_ex2(e.x), attn_ex2(e.y));
                        sum2[j & 1] = __fadd2_rn(sum2[j & 1], e);
                        if constexpr (BF16) {
                            const __nv_bfloat162 h = __floats2bfloat162_rn(e.x, e.y);
                            p[j] = *reinterpret_cast<const uint32_t *>(&h);
                        } else {
                            const __half2 h = __floats2half2_rn(e.x, e.y);
                            p[j] = *reinterpret_cast<const uint32_t *>(&h);
                        }
                    }
                    st32(col_p + N * c, p);
                    wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.p_full[q][c]);
                }
                sum += (sum2[0].x + sum2[0].y) + (sum2[1].x + sum2[1].y);
            }
            if (!ok) break;
            if (some) {
                ok = arrived(&sm.o_full[q], o_phase, a.status, abort_flag);
                if (!ok) break;
                o_phase ^= 1;
                tc_fence_after();
            }
            // What warp 10 has found was written before the unit's last values went to the MMAs.
            const bool spoilt = some && *const_cast<volatile uint32_t *>(&sm.spoilt[n & 15]) == n + 1;
            n += x.t1 > x.t0;
            const bool split = x.slot >= 0;
            uint8_t *dst = nullptr;
            if (live && split) {
                const int64_t slot = (int64_t)x.slot * ROWS + q * QROWS + row;
                a.ml[slot] = make_float2(at.mx, sum);
                dst = reinterpret_cast<uint8_t *>(a.part + slot * D);
            } else if (live) {
                const int tok = a.by_group(r);
                dst = static_cast<uint8_t *>(a.out) + ((x.row0 + tok) * a.ldo + (x.h * a.group + r - tok * a.group) * D) * out_size(a.otype);
            }
            // A row that sees nothing: 0.  A score times scale beyond f32: mx is infinite and so no weight counts, NaN (joined
            // parts, and warps in attention.cu, get it from the difference of two infinities).
            const float none = at.mx == -NEG ? NAN : 0.0f;
            const float inv = split ? 1.0f : sum == 0.0f ? none : 1.0f / sum;
            const int type = split ? Q8ACT_F32 : a.otype;
            uint8_t *out = smem + C::OFF_OUT + warp * OUT_BYTES;
#pragma unroll 1
            for (int i = 0; i < D; i += 64) {
                float o[64];
                if (some) {
                    ld32(col_o + i, o);
                    ld32(col_o + i + 32, o + 32);
                    wait_ld<64>(o);
                } else {
#pragma unroll
                    for (int j = 0; j < 64; ++j) o[j] = 0.0f;
                }
                if (spoilt && live) {
                    float e[64];
                    cleared_part<T, D>(a, x, q * QROWS + row, i, at.base(), e);
#pragma unroll
                    for (int j = 0; j < 64; ++j) o[j] += e[j];
                }
#pragma unroll
                for (int j = 0; j < 64; ++j) o[j] *= inv;
                uint4 v[8];
                if (type == Q8ACT_F32) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            v[k] = make_uint4(__float_as_uint(o[32 * h + 4 * k]), __float_as_uint(o[32 * h + 4 * k + 1]),
                                              __float_as_uint(o[32 * h + 4 * k + 2]), __float_as_uint(o[32 * h + 4 * k + 3]));
                        store_rows(out, v, dst, (i + 32 * h) * 4);
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        float f[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) f[j] = o[8 * k + j];
                        v[k] = type == Q8ACT_F16 ? pack<__half>(f) : pack<__nv_bfloat16>(f);
                    }
                    store_rows(out, v, dst, i * 2);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.unit_empty[round % RECORDS]);
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(OTHER_REGS));
        if (warp == 8) {
            // ------------------------------ MMA issuer ------------------------------
            uint32_t q_phase = 0, p_phase = 0, s_phase = 3, tiles = 0;      // a bit a row tile; tiles so far
            int st = 0;
            uint32_t phase = 0;
            bool ok = true;
            auto wait = [&](uint64_t *bar, uint32_t parity) { return ok = arrived(bar, parity, a.status, abort_flag); };
            const uint64_t qdesc = smem_desc_sw128(smem_u32(smem)), kdesc = smem_desc_sw128(smem_u32(stages));
            const uint64_t vdesc = smem_desc_mn_sw128(smem_u32(stages), C::HALF_BYTES);
            // This warp's instructions pace the tensor cores (it shares its scheduler with softmax warps): few waits, no
            // questions that can be spared.
            auto next = [&] {
                if (++st == STAGES) {
                    st = 0;
                    phase ^= 1;
                }
            };
            auto at = [&](uint64_t desc, int stage) { return desc + (uint32_t)(__shfl_sync(0xffffffffu, stage, 0) * (C::STAGE_BYTES >> 4)); };
            for (int round = 0; ok; ++round) {
                if (!wait(&sm.unit_full[round % RECORDS], round / RECORDS & 1)) break;
                // The same in all lanes to the compiler too: the loops then stay in uniform registers.
                struct { int t0, t1, a[2], b[2]; } rg;
                {
                    const Record &x = sm.units[round % RECORDS];
                    rg.t0 = __shfl_sync(0xffffffffu, x.t0, 0);
                    rg.t1 = __shfl_sync(0xffffffffu, x.t1, 0);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        rg.a[q] = __shfl_sync(0xffffffffu, x.a[q], 0);
                        rg.b[q] = __shfl_sync(0xffffffffu, x.b[q], 0);
                    }
                }
                if (rg.t0 < 0) break;
                if (lane == 0) mbar_arrive(&sm.unit_empty[round % RECORDS]);
                if (rg.t0 == rg.t1) continue;
                auto issue_qk = [&](int q, uint64_t kd) {
#pragma unroll
                    for (int i = 0; i < D / 16; ++i)
                        mma_ss(tmem + C::COL_S + q * TILE, qdesc + ((q * C::Q_BYTES + (i >> 2) * (QROWS * 128) + (i & 3) * 32) >> 4),
                               kd + ((i >> 2) * C::HALF_BYTES + (i & 3) * 32 >> 4), IDESC_QK, i > 0);
                };
                auto issue_pv = [&](int q, uint64_t vd, int from, int to, uint32_t add) {
#pragma unroll
                    for (int i = from; i < to; ++i)
                        mma_ts(tmem + C::COL_O + q * D, tmem + C::COL_P + q * C::P_STRIDE + 8 * i, vd + (i * 2048 >> 4), IDESC_PV,
                               i > 0 ? 1u : add);
                };
                // S = Q K^T of the tile whose keys are at kd.
                auto scores = [&](int q, int t, uint64_t kd) {
                    if (t < rg.a[q] || t >= rg.b[q]) return true;
                    if (t == rg.a[q]) {
                        if (!wait(&sm.q_full[q], q_phase >> q & 1)) return false;
                        q_phase ^= 1u << q;
                    }
                    if constexpr (C::OWN_P) {          // the last S (of the unit before, too) is in registers
                        if (!wait(&sm.s_empty[q], s_phase >> q & 1)) return false;
                        s_phase ^= 1u << q;
                    }
                    tc_fence_after();
                    if (elect_one()) {
                        issue_qk(q, kd);
                        tc_commit(&sm.s_full[q]);
                        if (t + 1 == rg.b[q]) tc_commit(&sm.q_empty[q]);
                    }
                    __syncwarp();
                    return true;
                };
                auto weighted = [&](int q, int t, uint64_t vd) {
                    if (t < rg.a[q] || t >= rg.b[q]) return true;
                    const uint32_t add = t > rg.a[q];
#pragma unroll
                    for (int part = 0; part < PARTS; ++part) {
                        constexpr int N = TILE / 16 / PARTS;
                        if (!wait(&sm.p_full[q][part], p_phase >> q & 1)) return false;
                        tc_fence_after();
                        if (elect_one()) {
                            issue_pv(q, vd, N * part, N * part + N, add);
                            if (C::OWN_P && part == PARTS - 1) tc_commit(&sm.p_empty[q]);
                            if (part == PARTS - 1 && t + 1 == rg.b[q]) tc_commit(&sm.o_full[q]);
                        }
                        __syncwarp();
                    }
                    p_phase ^= 1u << q;
                    return true;
                };
                auto release = [&](int stage) {
                    if (elect_one()) tc_commit(&sm.empty[stage]);
                    __syncwarp();
                };
                if (!wait(&sm.full[st], phase) || !scores(0, rg.t0, at(kdesc, st)) || !scores(1, rg.t0, at(kdesc, st))) break;
                release(st);
                next();
                if constexpr (C::OWN_P) {
                    uint64_t v_last = 0;
                    int st_last = 0;
                    for (int t = rg.t0; t <= rg.t1; ++t) {
                        const int vst = st;
                        int kst = st;
                        const bool here = t < rg.t1, more = t + 1 < rg.t1;
                        if (here) next();
                        kst = st;
                        if (more) next();
                        const uint64_t vd = at(vdesc, vst), kd = at(kdesc, kst);
                        if (here && !wait(&sm.ready[tiles & 7], tiles >> 3 & 1)) break;
                        tiles += here;
                        if (more && !scores(0, t + 1, kd)) break;
                        if (t > rg.t0) {
                            if (!weighted(1, t - 1, v_last)) break;
                            release(st_last);
                        }
                        if (more) {
                            if (!scores(1, t + 1, kd)) break;
                            release(kst);
                        }
                        if (here && !weighted(0, t, vd)) break;
                        v_last = vd;
                        st_last = vst;
                    }
                } else {
                    // Tiles that both row tiles take, with a next one that they take too, and neither's first or
                    // last but one: no questions asked.  (This warp's instructions pace the tensor cores.)
                    const int plain0 = max(rg.a[0], rg.a[1]) + 1, plain1 = min(rg.b[0], rg.b[1]) - 2;
                    for (int t = rg.t0; t < rg.t1; ++t, ++tiles) {
#pragma unroll 1
                        for (; t >= plain0 && t < plain1; ++t, ++tiles) {
                            const int vst = st;
                            next();
                            const int kst = st;
                            next();
                            const uint64_t vd = at(vdesc, vst), kd = at(kdesc, kst);
                            if (!wait(&sm.ready[tiles & 7], tiles >> 3 & 1)) break;
#pragma unroll
                            for (int q = 0; q < 2; ++q) {
#pragma unroll
                                for (int part = 0; part < PARTS; ++part) {
                                    constexpr int N = TILE / 16 / PARTS;
                                    if (!wait(&sm.p_full[q][part], p_phase >> q & 1)) break;
                                    tc_fence_after();
                                    if (elect_one()) {
                                        issue_pv(q, vd, N * part, N * part + N, 1u);
                                        if (part == PARTS - 1) {
                                            if (q == 1) tc_commit(&sm.empty[vst]);
                                            issue_qk(q, kd);
                                            tc_commit(&sm.s_full[q]);
                                            if (q == 1) tc_commit(&sm.empty[kst]);
                                        }
                                    }
                                    __syncwarp();
                                }
                                if (!ok) break;
                            }
                            p_phase ^= 3;
                            if (!ok) break;
                        }
                        if (!ok) break;
                        const int vst = st;
                        next();
                        const int kst = st;
                        const bool more = t + 1 < rg.t1;
                        if (more) next();
                        const uint64_t vd = at(vdesc, vst), kd = at(kdesc, kst);
                        if (!wait(&sm.ready[tiles & 7], tiles >> 3 & 1) || !weighted(0, t, vd)) break;
                        if (more && !scores(0, t + 1, kd)) break;
                        if (!weighted(1, t, vd)) break;
                        release(vst);
                        if (more) {
                            if (!scores(1, t + 1, kd)) break;
                            release(kst);
                        }
                    }
                }
            }
            if (!ok) {                   // MMAs may be in flight
                if (elect_one()) tc_commit(&sm.drained);
                __syncwarp();
                mbar_wait_drain(&sm.drained, 0, a.status);
            }
        } else if (warp == 9) {
            // ------------------------------ loader ------------------------------
            const int ps = 1 << a.p.page_shift, per_tile = ps < TILE ? TILE / ps : 1;
            int it = 0, st = 0;
            uint32_t phase = 1, tiles = 0;
            bool ok = true;
            for (int round = 0; ok; ++round) {
                ok = __all_sync(0xffffffffu, wait_or_abort(&sm.unit_full[round % RECORDS], round / RECORDS & 1, a.status, abort_flag));
                const Record &rc = sm.units[round % RECORDS];
                if (!ok || rc.t0 < 0) break;
                const int t0 = rc.t0, t1 = rc.t1, seq = rc.seq, h = rc.h;
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.unit_empty[round % RECORDS]);
                int64_t page = lane < per_tile && t0 < t1 ? page_of(a.p, seq, (t0 * TILE >> a.p.page_shift) + lane) : -1;
                for (int t = t0; ok && t < t1; ++t) {
                    const int pos = t * TILE;
                    // A page that does not exist: a box outside the tensor, which reads as zeros.
                    const int id = page < 0 ? (int)a.p.pages : (int)page;
                    const uint32_t good = __ballot_sync(0xffffffffu, page >= 0);
                    uint32_t pages = 0;
                    for (int j = 0; j < per_tile; ++j)
                        if (good >> j & 1) pages |= ((1u << (8 / per_tile)) - 1) << (j * (8 / per_tile));
                    if (t + 1 < t1 && lane < per_tile) page = page_of(a.p, seq, ((pos + TILE) >> a.p.page_shift) + lane);
                    for (int kv = 0; kv < 2; ++kv, ++it) {
                        ok = __all_sync(0xffffffffu, wait_or_abort(&sm.empty[st], phase, a.status, abort_flag));
                        if (!ok) break;
                        if (lane == 0) {
                            if (kv == 0) *const_cast<volatile uint32_t *>(&sm.pages[tiles++ & 7]) = pages;
                            mbar_arrive_expect_tx(&sm.full[st], C::STAGE_BYTES);
                        }
                        __syncwarp();
                        const int j = lane / C::HALVES, half = lane % C::HALVES;
                        const int box_page = __shfl_sync(0xffffffffu, id, j & 31);
                        if (j < per_tile)
                            tma_load_4d(stages + st * C::STAGE_BYTES + half * C::HALF_BYTES + j * ps * 128, kv ? &tm_v : &tm_k,
                                        half * 64, ps > TILE ? pos & (ps - 1) : 0, h, box_page, &sm.full[st]);
                        __syncwarp();
                        if (++st == STAGES) {
                            st = 0;
                            phase ^= 1;
                        }
                    }
                }
            }
            // Never leave with a copy into this CTA's shared memory in flight.
            for (int i = it > STAGES ? it - STAGES : 0; i < it; ++i)
                mbar_wait_drain(&sm.full[i % STAGES], (i / STAGES) & 1, a.status);
        } else if (warp == 10) {
            // ------------------------------ masked values ------------------------------
            int st = 0;
            uint32_t phase = 0, n = 0, tiles = 0;
            bool ok = true;
            for (int round = 0; ok; ++round) {
                ok = __all_sync(0xffffffffu, wait_or_abort(&sm.unit_full[round % RECORDS], round / RECORDS & 1, a.status, abort_flag));
                const Record &x = sm.units[round % RECORDS];
                if (!ok || x.t0 < 0) break;
                // Every stage is waited for and handed back, so that this warp keeps the pipeline's pace.
                for (int i = 0; i < 2 * (x.t1 - x.t0); ++i) {
                    const int t = x.t0 + (i >> 1);
                    ok = __all_sync(0xffffffffu, wait_or_abort(&sm.full[st], phase, a.status, abort_flag));
                    if (!ok) break;
                    if ((i & 1) && x.masked(a, t)) {
                        // Positions of the tile that not all rows see: before `from`, behind the window, and from
                        // `to` on.
                        const int k0 = t * TILE;
                        const int to = min(max(min(x.first, x.hi) + 1 - k0, 0), TILE);
                        const int from = min(max(a.window ? x.last - a.window + 1 : 0, x.lo) - k0, TILE);
                        const bool found = fix_rows<T, D>(stages + st * C::STAGE_BYTES, 0, from, x.lo - k0, x.hi - k0) |
                                           fix_rows<T, D>(stages + st * C::STAGE_BYTES, max(to, from), TILE, x.lo - k0, x.hi - k0);
                        if (__any_sync(0xffffffffu, found)) {
                            clear_non_finite<T, D>(stages + st * C::STAGE_BYTES, x.lo - k0, x.hi - k0, from, to);
                            if (lane == 0) *const_cast<volatile uint32_t *>(&sm.spoilt[n & 15]) = n + 1;
                        }
                        fence_proxy_async_smem();
                    }
                    __syncwarp();
                    if (lane == 0) {
                        // Values and the next keys are there (the last values: no keys follow).
                        if (i > 0 && (!(i & 1) || t + 1 == x.t1)) mbar_arrive(&sm.ready[tiles++ & 7]);
                        mbar_arrive(&sm.empty[st]);
                    }
                    if (++st == STAGES) {
                        st = 0;
                        phase ^= 1;
                    }
                }
                n += x.t1 > x.t0;
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.unit_empty[round % RECORDS]);
            }
        } else {
            // ------------------------------ units, queries ------------------------------
            Plan<ROWS, TILE, FEW> plan;
            plan.make(a);
            uint32_t q_phase = 3, q_loads = 0;               // a bit a row tile
            bool ok = true;
            for (int round = 0;; ++round) {
                if (!__all_sync(0xffffffffu, wait_or_abort(&sm.unit_empty[round % RECORDS], (round / RECORDS & 1) ^ 1, a.status, abort_flag)))
                    break;
                const int64_t u = unit_of(round);
                Record rc;
                rc.t0 = -1;
                if (u < plan.total) {
                    const Unit x = plan.find(a, (int)u);
                    rc.rows = x.s.n * a.group;
                    rc.r0 = x.tile * ROWS;
                    const int r1 = min(rc.r0 + ROWS, rc.rows) - 1;
                    const Span s = span_of<TILE>(a, x.s, rc.r0, r1);
                    s.part(x.part, x.parts, rc.t0, rc.t1);
                    rc.lo = s.lo;
                    rc.hi = s.hi;
                    rc.first = x.s.pos0 + a.by_group(rc.r0);
                    rc.last = x.s.pos0 + a.by_group(r1);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const int q0 = rc.r0 + q * QROWS;
                        rc.a[q] = rc.b[q] = rc.t0;
                        if (q0 <= r1) {
                            const Span z = span_of<TILE>(a, x.s, q0, min(q0 + QROWS - 1, r1));
                            rc.a[q] = max(rc.t0, z.first);
                            rc.b[q] = max(rc.a[q], min(rc.t1, z.first + z.n));
                        }
                    }
                    rc.row0 = x.s.row0;
                    rc.h = x.h;
                    rc.pos0 = x.s.pos0;
                    rc.end = x.s.end;
                    rc.seq = x.b;
                    rc.slot = x.parts > 1 ? x.slot + x.part : -1;
                }
                if (lane == 0) {
                    sm.units[round % RECORDS] = rc;
                    mbar_arrive(&sm.unit_full[round % RECORDS]);
                }
                if (rc.t0 < 0) break;
                for (int q = 0; q < 2; ++q) {
                    if (q ? rc.b[1] <= rc.a[1] : rc.b[0] <= rc.a[0]) continue;
                    ok = __all_sync(0xffffffffu, wait_or_abort(&sm.q_empty[q], q_phase >> q & 1, a.status, abort_flag));
                    if (!ok) break;
                    q_phase ^= 1u << q;
                    if constexpr (BOXES) {
                        // Whole tokens: a box of a row tile's.  (Rows behind the sequence's last hold others' queries,
                        // or zeros; what comes of them goes nowhere.)
                        if (lane == 0) {
                            mbar_arrive_expect_tx(&sm.q_full[q], C::Q_BYTES);
                            for (int half = 0; half < C::HALVES; ++half)
                                tma_load_3d(smem + q * C::Q_BYTES + half * (QROWS * 128), &tm_q, half * 64, rc.h * a.group,
                                            rc.row0 + a.by_group(rc.r0 + q * QROWS), &sm.q_full[q]);
                        }
                        __syncwarp();
                        q_loads |= 1u << q;
                    } else {
                        // Rows behind the last one as zeros, or, of whole warps of them, as they were.
                        const int rows = rc.rows, r0 = rc.r0 + q * QROWS;
                        constexpr int VECS = D / 8, AT_ONCE = 32 / VECS;       // 16-byte vectors of a row, rows a round of lanes
                        const uint32_t dst0 = smem_u32(smem + q * C::Q_BYTES);
#pragma unroll 1
                        for (int i = 0; i < min(QROWS, rows - r0); i += 32) {
                            const int r = r0 + i + lane, tok = a.by_group(r);
                            const int64_t off = r < rows ? (rc.row0 + tok) * a.ldq + (rc.h * a.group + r - tok * a.group) * D : -1;
#pragma unroll 8
                            for (int j = 0; j < 32; j += AT_ONCE) {
                                const int rr = i + j + lane / VECS, v = lane % VECS;
                                const int64_t o = __shfl_sync(0xffffffffu, off, j + lane / VECS);
                                cp_async16(dst0 + (v >> 3) * (QROWS * 128) + rr * 128 + (((v & 7) ^ (rr & 7)) << 4),
                                           static_cast<const T *>(a.q) + (o < 0 ? 0 : o) + v * 8, o < 0 ? 0 : 16);
                            }
                        }
                        asm volatile("cp.async.wait_all;" ::: "memory");
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sm.q_full[q]);
                    }
                }
                if (!ok) break;
            }
            // Never leave with a copy into this CTA's shared memory in flight: the last unit's queries (of the units
            // before, the MMAs have waited for them).
            if (BOXES)
                for (int q = 0; q < 2; ++q)
                    if (q_loads >> q & 1) mbar_wait_drain(&sm.q_full[q], q_phase >> q & 1, a.status);
        }
    }
    __syncthreads();
    if (warp == 8) tc_dealloc(tmem, 512);
}

}  // namespace

// Partial results: of three rounds of a GB300's 152 SMs.
constexpr int SLOTS = 3 * 152;

size_t attention_chunk_space(int dim) { return attention_space(SLOTS, ROWS, dim); }

cudaError_t launch_attention_chunk(const DeviceInfo &dev, const q8act_paged_kv &kv, Attn a, void *ws, cudaStream_t stream)
{
    attention_place(a, ws, SLOTS, ROWS);
    a.ctas = dev.num_sms;
    a.least = 2;
    // 128 values a head, f16: 509 tokens at 16384 (32 + 8 heads) 4 cuts each row tile in 7 and takes 116 us, 8 and 16 in 2: 101; 200 at
    // 30000 2: 109, 4: 97, 8 and 16: 90.  64 values: 2, 4, 8 and 16 within 1.5 % of each other (509 at 16384, 64 + 8 heads 148, 20 + 4
    // heads 60.5; 200 at 30000, 12 + 12 heads 36; window, verification and mixed batches, too).
    a.unit_cost = 8.0f;
    CUtensorMap tk, tv, tq;
    if (!attention_maps(kv, TILE, &tk, &tv)) return cudaErrorInvalidValue;
    const bool q_boxes = QROWS % a.group == 0;
    if (q_boxes) {
        const uint64_t dims[3] = {(uint64_t)kv.dim, (uint64_t)a.group * kv.heads, (uint64_t)a.p.m};
        const uint64_t strides[2] = {(uint64_t)kv.dim * 2, (uint64_t)a.ldq * 2};
        const uint32_t box[3] = {64, (uint32_t)a.group, (uint32_t)(QROWS / a.group)};
        if (!encode_tiled(&tq, attention_type(kv), a.q, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B)) return cudaErrorInvalidValue;
    } else {
        tq = tk;
    }
    return with_type(kv.type, [&](auto x) -> cudaError_t {
        using T = decltype(x);
        if constexpr (sizeof(T) == 4) {
            return cudaErrorInvalidValue;
        } else {
            auto go = [&](auto d, auto few, auto boxes) -> cudaError_t {
                constexpr int D = decltype(d)::value;
                constexpr bool FEW = decltype(few)::value, BOXES = decltype(boxes)::value;
                constexpr size_t smem = Cfg<D>::OFF_SHARED + sizeof(Shared);
                static_assert(smem <= 227 * 1024, "shared memory");
                cudaError_t e = set_kernel_smem<attention_chunk_kernel<T, D, FEW, BOXES>>(dev.device, smem);
                if (e != cudaSuccess) return e;
                e = launch_dependent(attention_chunk_kernel<T, D, FEW, BOXES>, dim3(a.ctas), THREADS, smem, stream, tk, tv, tq, a);
                return e == cudaSuccess ? launch_attention_chunk_join(dev, a, D, stream) : e;
            };
            auto by_queries = [&](auto d, auto few) { return q_boxes ? go(d, few, std::true_type{}) : go(d, few, std::false_type{}); };
            auto pick = [&](auto d) { return kv.seqs <= 32 ? by_queries(d, std::true_type{}) : by_queries(d, std::false_type{}); };
            return kv.dim == 64 ? pick(std::integral_constant<int, 64>{}) : pick(std::integral_constant<int, 128>{});
        }
    });
}

}  // namespace q8
