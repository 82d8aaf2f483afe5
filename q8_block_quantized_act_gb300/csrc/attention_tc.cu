// attention_tc.cu -- attention of chunks of new tokens over a paged cache on the tensor cores (tcgen05).
//   S = Q K^T,  P = e^(scale S - mx),  O = P V,  out = O / sum P
//
// A CTA holds two tiles of 128 rows (query heads of a group x tokens) and walks over tiles of 128
// positions.  S and O are accumulators in tensor memory; P, rounded to the cache's type, takes the place
// of S there and is the second product's first operand, so only Q, K and V go through shared memory.
// While the four warps of one row tile turn S into P, the tensor cores work for the other tile.
//   warps 0-3, 4-7  a row tile each: a thread a row, so maxima and sums need no exchange
//   warp 8          issues the MMAs: P0 V, Q0 K', P1 V, Q1 K' (K' the next tile's keys)
//   warp 9          brings pages of keys and values to shared memory (TMA, 128-byte swizzled)
//   warps 10, 11    bring a row tile's queries each; in tiles of values that some row does not see as a whole they
//                   clear those that no row sees and look for infinities and NaN among the others (attention.cuh)
// O is rescaled only when a row's maximum has risen by more than 2^8 since the last time: until then P is
// at most 2^8 and nothing is lost (f32 sums, the type's relative precision).
#include <algorithm>

#include "attention.cuh"

namespace q8 {
namespace {

constexpr int TILE = 128;                // positions a step
constexpr int QROWS = 128;               // rows of a row tile
constexpr int ROWS = CHUNK_ROWS;         // of a unit: two row tiles
constexpr int COUNTERS = 64;             // threads that count the units
constexpr int THREADS = 384;
constexpr int SOFTMAX_REGS = 208, OTHER_REGS = 88;      // 256 x 208 + 128 x 88 = 384 x 168, the launch's registers
constexpr int PARTS = 2;                 // of a tile's weights, handed to the MMAs one by one
constexpr float NEG = -INFINITY;
constexpr float SLACK = 8.0f;

template <int D>
struct Cfg {
    static constexpr int Q_BYTES = QROWS * D * 2;              // a row tile's queries
    static constexpr int STAGE_BYTES = TILE * D * 2;           // a tile of keys or of values
    static constexpr int STAGES = 160 * 1024 / STAGE_BYTES;
    static constexpr int HALVES = D / 64;                      // columns of 128 bytes
    static constexpr int HALF_BYTES = TILE * 128;
    static constexpr int STAGES_END = 2 * Q_BYTES + STAGES * STAGE_BYTES;
    static constexpr uint32_t COL_S = 0, COL_O = 2 * TILE;     // tensor memory: S0 S1 O0 O1
    // Instruction descriptor, kind::f16: D f32 (bits 4-5), types of A and B (7-9, 10-12), B's major (16; 1: its
    // rows are K), N >> 3 (17-22), M >> 4 (24-28).
    static constexpr uint32_t IDESC_QK = (1u << 4) | ((uint32_t)(TILE >> 3) << 17) | ((uint32_t)(QROWS >> 4) << 24);
    static constexpr uint32_t IDESC_PV = (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | ((uint32_t)(QROWS >> 4) << 24);
    static constexpr uint32_t IDESC_BF16 = (1u << 7) | (1u << 10);
};

struct Shared {
    PlanSmem<COUNTERS> plan;
    uint64_t full[10], empty[10];                    // stages
    // Tile n of the CTA, in barrier n % 8: its values, and the next tile's keys, are there.  The stages hold five tiles
    // at most, so six barriers would do.
    uint64_t ready[8];
    uint64_t s_full[2], p_full[2][PARTS], q_full[2], q_empty[2], o_full[2], drained;
    uint32_t pages[8];                               // tile n of the CTA in word n % 8: its 16-position blocks whose page exists
    uint32_t tmem;
    // Unit n of the CTA, counting those with positions, has a non-finite value that not all rows see: n + 1 in word
    // n % 16.  Warps 10 and 11 are ahead of the softmax by the stages' tiles at most, 5 and one.
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
__device__ __forceinline__ void st16(uint32_t taddr, const uint32_t *u)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
        ::"r"(taddr), "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]),
          "r"(u[9]), "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15])
        : "memory");
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
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 16 bytes from global to shared memory, of which the first `bytes` are read and the others zeros.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint32_t bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// 64 bytes of each lane's row at `off`, four lanes to a row at a time: a store then touches 8 rows, not 32, and
// whole sectors of them.  rows: of the quad's lanes (null: not stored).
__device__ __forceinline__ void quad_store(uint4 (&v)[4], uint8_t *const (&rows)[4], int off)
{
    const int lane = threadIdx.x & 3;
    uint32_t(*w)[4] = reinterpret_cast<uint32_t(*)[4]>(v);
#pragma unroll
    for (int bit = 1; bit < 4; bit <<= 1)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i & bit) continue;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t got = __shfl_xor_sync(0xffffffffu, lane & bit ? w[i][k] : w[i | bit][k], bit);
                if (lane & bit) w[i][k] = got;
                else w[i | bit][k] = got;
            }
        }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (rows[i]) *reinterpret_cast<uint4 *>(rows[i] + off + lane * 16) = v[i];
}

// 32 consecutive values of each lane's row, from value `at` on, rounded to `type`.
__device__ __forceinline__ void store32(uint8_t *const (&rows)[4], int type, int at, const float (&v)[32])
{
    uint4 w[4];
    if (type == Q8ACT_F32) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[j] = make_uint4(__float_as_uint(v[16 * h + 4 * j]), __float_as_uint(v[16 * h + 4 * j + 1]),
                                  __float_as_uint(v[16 * h + 4 * j + 2]), __float_as_uint(v[16 * h + 4 * j + 3]));
            quad_store(w, rows, (at + 16 * h) * 4);
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = v[8 * j + i];
        w[j] = type == Q8ACT_F16 ? pack<__half>(f) : pack<__nv_bfloat16>(f);
    }
    quad_store(w, rows, at * 2);
}

// A unit's tiles: [t0, t1), and those that row tile q sees, [a[q], b[q]).
struct Range {
    int t0, t1, a[2], b[2];
    int lo, hi;              // positions that at least one row sees
    int first, last;         // positions of the first and the last row

    __device__ __forceinline__ Range(const Attn &at, const Unit &x)
    {
        const int rows = x.s.n * at.group, r0 = x.tile * ROWS, r1 = min(r0 + ROWS, rows) - 1;
        const Span s = span_of<TILE>(at, x.s, r0, r1);
        s.part(x.part, x.parts, t0, t1);
        lo = s.lo;
        hi = s.hi;
        first = x.s.pos0 + at.by_group(r0);
        last = x.s.pos0 + at.by_group(r1);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int q0 = r0 + q * QROWS;
            a[q] = b[q] = t0;
            if (q0 <= r1) {
                const Span z = span_of<TILE>(at, x.s, q0, min(q0 + QROWS - 1, r1));
                a[q] = max(t0, z.first);
                b[q] = max(a[q], min(t1, z.first + z.n));
            }
        }
    }
    // The same in all lanes to the compiler too: the MMA warp's loops then stay in uniform registers.
    __device__ __forceinline__ void uniform()
    {
        int *v[] = {&t0, &t1, &a[0], &a[1], &b[0], &b[1], &lo, &hi, &first, &last};
#pragma unroll
        for (int *i : v) *i = __shfl_sync(0xffffffffu, *i, 0);
    }
    // Whether some row does not see some of a tile.
    __device__ __forceinline__ bool masked(const Attn &at, int t) const
    {
        return t * TILE < lo || t * TILE + TILE - 1 > min(first, hi) || (at.window && t * TILE <= last - at.window);
    }
};

// The unit of this CTA's round: rounds run forwards and backwards in turn, since earlier units are longer.
__device__ __forceinline__ int64_t unit_of(int round)
{
    const int c = blockIdx.x, g = gridDim.x;
    return (int64_t)round * g + (round & 1 ? g - 1 - c : c);
}

// Columns c0 .. c0 + 31 of each lane's row's sums, taken again (attention.cuh).
template <typename T, int D>
__device__ __noinline__ void exact_part(const Attn &a, const Plan<ROWS, TILE, COUNTERS> &plan, const PlanSmem<COUNTERS> &sm, int u,
                                        int row, bool live, int c0, float mx, float (&o)[32])
{
    const Unit x = plan.find(a, sm, u);
    if (!live) return;
    const Range rg(a, x);
    const int r = x.tile * ROWS + row, tok = a.by_group(r), pos = x.s.pos0 + tok;
    const int k0 = max(a.window ? pos - a.window + 1 : 0, rg.t0 * TILE), k1 = min(min(pos, x.s.end - 1), rg.t1 * TILE - 1);
    exact_values<T, D>(a, x.b, x.h, static_cast<const T *>(a.q) + (x.s.row0 + tok) * a.ldq + (x.h * a.group + r - tok * a.group) * D,
                       k0, k1, mx == NEG ? 0.0f : mx, [&](int j) { return c0 + j; }, o);
}

template <typename T, int D>
__global__ void __launch_bounds__(THREADS, 1)
    attention_chunk_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, Attn a)
{
    using C = Cfg<D>;
    constexpr bool BF16 = std::is_same<T, __nv_bfloat16>::value;
    constexpr int STAGES = C::STAGES;
    constexpr uint32_t IDESC_QK = C::IDESC_QK | (BF16 ? C::IDESC_BF16 : 0), IDESC_PV = C::IDESC_PV | (BF16 ? C::IDESC_BF16 : 0);
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *stages = smem + 2 * C::Q_BYTES;
    Shared &sm = *reinterpret_cast<Shared *>(smem + C::STAGES_END);
    volatile int *abort_flag = &sm.abort_flag;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) { mbar_init(&sm.full[s], 1); mbar_init(&sm.empty[s], 3); }
        for (int i = 0; i < 8; ++i) mbar_init(&sm.ready[i], 2);
        for (int q = 0; q < 2; ++q) {
            mbar_init(&sm.s_full[q], 1);
            for (int i = 0; i < PARTS; ++i) mbar_init(&sm.p_full[q][i], 4);
            mbar_init(&sm.q_full[q], 1);
            mbar_init(&sm.q_empty[q], 1);
            mbar_init(&sm.o_full[q], 1);
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
    }
    griddep_wait();
    griddep_launch_dependents();
    Plan<ROWS, TILE, COUNTERS> plan;
    tc_fence_before();
    plan.make(a, sm.plan);                           // its barriers: the ones above exist for all
    tc_fence_after();
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.count = sm.plan.items[COUNTERS];
    const uint32_t tmem = __shfl_sync(0xffffffffu, sm.tmem, 0);

    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(SOFTMAX_REGS));
        // ------------------------------ softmax ------------------------------
        const int q = warp >> 2, row = (warp & 3) * 32 + lane;         // of the row tile
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;             // the warp's lanes of tensor memory
        const uint32_t col_s = tmem + lanes + C::COL_S + q * TILE, col_o = tmem + lanes + C::COL_O + q * D;
        uint32_t s_phase = 0, o_phase = 0, n = 0, tiles = 0;
        bool ok = true;
        struct Work {
            int64_t u;                         // the unit, or beyond the last
            int t, end;                        // tiles of the row tile
            int from, count;                   // the unit's first tile and how many
            int hi, lo;                        // positions that the row sees
            bool live;
            int64_t slot;                      // of the row in the partial results, or -1
            uint8_t *dst;                      // where the row goes, or null
        };
        auto enter = [&](int64_t u) {
            Work w;
            w.u = u;
            if (u >= plan.total) return w;
            const Unit x = plan.find(a, sm.plan, (int)u);
            const Range rg(a, x);
            const int rows = x.s.n * a.group, r = x.tile * ROWS + q * QROWS + row;
            w.t = rg.a[q];
            w.end = rg.b[q];
            w.from = rg.t0;
            w.count = rg.t1 - rg.t0;
            w.live = r < rows;
            const int tok = w.live ? a.by_group(r) : 0, pos = x.s.pos0 + tok;
            w.hi = w.live ? min(pos, x.s.end - 1) : INT_MAX;
            w.lo = w.live && a.window ? max(pos - a.window + 1, 0) : 0;
            w.slot = -1;
            w.dst = nullptr;
            if (x.parts > 1) {
                if (x.part == 0 && threadIdx.x == 0)
                    a.items[x.item] = Item{x.slot, x.parts, x.s.row0, x.tile * ROWS, x.h, min(ROWS, rows - x.tile * ROWS), {0, 0}};
                if (w.live) {
                    w.slot = (int64_t)(x.slot + x.part) * ROWS + q * QROWS + row;
                    w.dst = reinterpret_cast<uint8_t *>(a.part + w.slot * D);
                }
            } else if (w.live) {
                w.dst = static_cast<uint8_t *>(a.out) +
                        ((x.s.row0 + tok) * a.ldo + (x.h * a.group + r - tok * a.group) * D) * out_size(a.otype);
            }
            return w;
        };
        Work w = enter(unit_of(0));
        for (int round = 1; w.u < plan.total; ++round) {
            const int hi = w.hi, lo = w.lo, end = w.end;
            const bool some = end > w.t;
            tiles -= w.from;                   // tile t of the sequence is tile tiles + t of the CTA
            bool first = true;
            float mx = NEG, sum = 0.0f;
            for (int t = w.t; t < end; ++t) {
                ok = __all_sync(0xffffffffu, wait_or_abort(&sm.s_full[q], s_phase, a.status, abort_flag));
                if (!ok) break;
                s_phase ^= 1;
                tc_fence_after();
                float s[TILE];
#pragma unroll
                for (int i = 0; i < TILE / 32; ++i) ld32(col_s + 32 * i, s + 32 * i);
                const int k0 = t * TILE;
                const uint32_t pages = *const_cast<volatile uint32_t *>(&sm.pages[(tiles + t) & 7]);
                const bool edge = __any_sync(0xffffffffu, k0 + TILE - 1 > hi || k0 < lo) || pages != 0xff;
                wait_ld<TILE>(s);
                if (edge) {
                    const int from = lo - k0, to = hi - k0;
#pragma unroll
                    for (int j = 0; j < TILE; ++j)
                        if (j < from || j > to || !(pages >> (j / 16) & 1)) s[j] = NEG;
                }
                float m4[4] = {NEG, NEG, NEG, NEG};
#pragma unroll
                for (int j = 0; j < TILE; j += 8)
#pragma unroll
                    for (int i = 0; i < 4; ++i) m4[i] = fmaxf(fmaxf(m4[i], s[j + 2 * i]), s[j + 2 * i + 1]);
                const float m = fmaxf(mx, fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * a.scale);
                if (first) {
                    mx = m;
                    first = false;
                } else if (__any_sync(0xffffffffu, m > mx + SLACK)) {
                    // (mx may be -inf: nothing seen so far, O and the sum are zeros)
                    const float f = attn_ex2(mx - (m == NEG ? 0.0f : m));
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
                    mx = m;
                }
                const float base = mx == NEG ? 0.0f : mx;
                const float2 scale2 = make_float2(a.scale, a.scale), base2 = make_float2(-base, -base);
                float2 sum2[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
                for (int i = 0; i < PARTS; ++i) {
#pragma unroll
                    for (int h = 0; h < 4 / PARTS; ++h) {
                        const int at = 32 * (4 / PARTS * i + h);
                        uint32_t p[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            float2 e = __ffma2_rn(make_float2(s[at + 2 * j], s[at + 2 * j + 1]), scale2, base2);
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
                        st16(col_s + at / 2, p);
                    }
                    wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.p_full[q][i]);
                }
                sum += (sum2[0].x + sum2[0].y) + (sum2[1].x + sum2[1].y);
            }
            if (!ok) break;
            tiles += w.from + w.count;
            // The next unit while the last products run.
            const Work next = enter(unit_of(round));
            if (some) {
                ok = __all_sync(0xffffffffu, wait_or_abort(&sm.o_full[q], o_phase, a.status, abort_flag));
                if (!ok) break;
                o_phase ^= 1;
                tc_fence_after();
            }
            // What warps 10 and 11 have found was written before the unit's last values went to the MMAs.
            const bool spoilt = some && *const_cast<volatile uint32_t *>(&sm.spoilt[n & 15]) == n + 1;
            n += w.count > 0;
            const bool split = w.slot >= 0;
            if (split) a.ml[w.slot] = make_float2(mx, sum);
            const float inv = split ? 1.0f : sum == 0.0f ? 0.0f : 1.0f / sum;          // a row that sees nothing: 0
            // (rows that are not there follow their warp's first, which decides the type)
            const int type = __any_sync(0xffffffffu, split) ? Q8ACT_F32 : a.otype;
            uint8_t *rows[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                rows[i] = reinterpret_cast<uint8_t *>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(w.dst), (lane & ~3) + i));
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                float o[32];
                if (some) {
                    ld32(col_o + 32 * i, o);
                    wait_ld<32>(o);
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) o[j] = 0.0f;
                }
                if (spoilt) {
                    float e[32];
                    exact_part<T, D>(a, plan, sm.plan, (int)w.u, q * QROWS + row, w.live, 32 * i, mx, e);
#pragma unroll
                    for (int j = 0; j < 32; ++j) o[j] = e[j];
                }
#pragma unroll
                for (int j = 0; j < 32; ++j) o[j] *= inv;
                store32(rows, type, 32 * i, o);
            }
            w = next;
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(OTHER_REGS));
        if (warp == 8) {
            // ------------------------------ MMA issuer ------------------------------
            uint32_t q_phase = 0, p_phase = 0, tiles = 0;           // a bit a row tile; tiles so far
            int st = 0;
            uint32_t phase = 0;
            bool ok = true;
            const uint64_t qdesc = smem_desc_sw128(smem_u32(smem)), kdesc = smem_desc_sw128(smem_u32(stages));
            const uint64_t vdesc = smem_desc_mn_sw128(smem_u32(stages), C::HALF_BYTES);
            // This warp's instructions pace the tensor cores (it shares its scheduler with softmax warps), so a wait
            // that is over takes one look, and there are few of them.
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                if (!__all_sync(0xffffffffu, mbar_try_wait(bar, parity)))
                    ok = __all_sync(0xffffffffu, wait_or_abort(bar, parity, a.status, abort_flag));
                return ok;
            };
            auto next = [&] {
                if (++st == STAGES) {
                    st = 0;
                    phase ^= 1;
                }
            };
            auto at = [&](uint64_t desc, int stage) { return desc + (uint32_t)(__shfl_sync(0xffffffffu, stage, 0) * (C::STAGE_BYTES >> 4)); };
            for (int round = 0; ok; ++round) {
                const int64_t u = unit_of(round);
                if (u >= plan.total) break;
                Range rg(a, plan.find(a, sm.plan, (int)u));
                rg.uniform();
                if (rg.t0 == rg.t1) continue;
                // S = Q K^T of the tile whose keys are at kd.
                auto scores = [&](int q, int t, uint64_t kd) {
                    if (t < rg.a[q] || t >= rg.b[q]) return true;
                    if (t == rg.a[q]) {
                        if (!wait(&sm.q_full[q], q_phase >> q & 1)) return false;
                        q_phase ^= 1u << q;
                    }
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int i = 0; i < D / 16; ++i)
                            mma_ss(tmem + C::COL_S + q * TILE, qdesc + ((q * C::Q_BYTES + (i >> 2) * (QROWS * 128) + (i & 3) * 32) >> 4),
                                   kd + ((i >> 2) * C::HALF_BYTES + (i & 3) * 32 >> 4), IDESC_QK, i > 0);
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
#pragma unroll
                            for (int i = N * part; i < N * part + N; ++i)
                                mma_ts(tmem + C::COL_O + q * D, tmem + C::COL_S + q * TILE + 8 * i, vd + (i * 2048 >> 4), IDESC_PV,
                                       i > 0 ? 1u : add);
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
                for (int t = rg.t0; t < rg.t1; ++t, ++tiles) {
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
                const int64_t u = unit_of(round);
                if (u >= plan.total) break;
                const Unit x = plan.find(a, sm.plan, (int)u);
                const Range rg(a, x);
                int64_t page = lane < per_tile && rg.t0 < rg.t1 ? page_of(a.p, x.b, (rg.t0 * TILE >> a.p.page_shift) + lane) : -1;
                for (int t = rg.t0; ok && t < rg.t1; ++t) {
                    const int pos = t * TILE;
                    // A page that does not exist: a box outside the tensor, which reads as zeros.
                    const int id = page < 0 ? (int)a.p.pages : (int)page;
                    const uint32_t good = __ballot_sync(0xffffffffu, page >= 0);
                    uint32_t pages = 0;
                    for (int j = 0; j < per_tile; ++j)
                        if (good >> j & 1) pages |= ((1u << (8 / per_tile)) - 1) << (j * (8 / per_tile));
                    if (t + 1 < rg.t1 && lane < per_tile) page = page_of(a.p, x.b, ((pos + TILE) >> a.p.page_shift) + lane);
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
                                        half * 64, ps > TILE ? pos & (ps - 1) : 0, x.h, box_page, &sm.full[st]);
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
        } else {
            // ------------------------------ masked values ------------------------------
            constexpr uint32_t E = BF16 ? 0x7f80u : 0x7c00u;
            const int q = warp - 10;                 // row tile whose queries it brings, half of a tile that it looks at
            int st = 0;
            uint32_t phase = 0, q_phase = 1, n = 0, tiles = 0;
            bool ok = true;
            for (int round = 0; ok; ++round) {
                const int64_t u = unit_of(round);
                if (u >= plan.total) break;
                const Unit x = plan.find(a, sm.plan, (int)u);
                const Range rg(a, x);
                if (rg.b[q] > rg.a[q]) {
                    ok = __all_sync(0xffffffffu, wait_or_abort(&sm.q_empty[q], q_phase, a.status, abort_flag));
                    if (!ok) break;
                    q_phase ^= 1;
                    // Rows behind the last one as zeros.
                    const int rows = x.s.n * a.group, r0 = x.tile * ROWS + q * QROWS;
                    constexpr int VECS = D / 8, AT_ONCE = 32 / VECS;       // 16-byte vectors of a row, rows a round of lanes
                    const uint32_t dst0 = smem_u32(smem + q * C::Q_BYTES);
#pragma unroll 1
                    for (int i = 0; i < QROWS; i += 32) {
                        const int r = r0 + i + lane, tok = a.by_group(r);
                        const int64_t off = r < rows ? (x.s.row0 + tok) * a.ldq + (x.h * a.group + r - tok * a.group) * D : -1;
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
                // Every stage is waited for and handed back, so that these warps keep the pipeline's pace.
                for (int i = 0; i < 2 * (rg.t1 - rg.t0); ++i) {
                    const int t = rg.t0 + (i >> 1);
                    ok = __all_sync(0xffffffffu, wait_or_abort(&sm.full[st], phase, a.status, abort_flag));
                    if (!ok) break;
                    if ((i & 1) && rg.masked(a, t)) {
                        bool found = false;
                        uint8_t *v = stages + st * C::STAGE_BYTES;
#pragma unroll 4
                        for (int j = q * 32 + lane; j < C::STAGE_BYTES / 16; j += 64) {
                            const int key = t * TILE + (j >> 3) % TILE;          // 8 vectors a position and half
                            uint4 *p = reinterpret_cast<uint4 *>(v) + j;
                            if (key < rg.lo || key > rg.hi) {
                                *p = make_uint4(0, 0, 0, 0);
                            } else {
                                const uint4 w = *p;
                                const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                                for (int l = 0; l < 4; ++l) found |= (ws[l] & E) == E || (ws[l] >> 16 & E) == E;
                            }
                        }
                        if (found) *const_cast<volatile uint32_t *>(&sm.spoilt[n & 15]) = n + 1;
                        fence_proxy_async_smem();
                    }
                    __syncwarp();
                    if (lane == 0) {
                        // Values and the next keys are there (the last values: no keys follow).
                        if (i > 0 && (!(i & 1) || t + 1 == rg.t1)) mbar_arrive(&sm.ready[tiles++ & 7]);
                        mbar_arrive(&sm.empty[st]);
                    }
                    if (++st == STAGES) {
                        st = 0;
                        phase ^= 1;
                    }
                }
                n += rg.t1 > rg.t0;
            }
        }
    }
    __syncthreads();
    if (warp == 8) tc_dealloc(tmem, 512);
}

}  // namespace

// A part for each of a GB300's 152 SMs.
constexpr int TARGET = 152;

size_t attention_chunk_space(int dim) { return attention_space(TARGET, ROWS, dim); }

cudaError_t launch_attention_chunk(const DeviceInfo &dev, const q8act_paged_kv &kv, Attn a, void *ws, cudaStream_t stream)
{
    attention_place(a, ws, TARGET, ROWS);
    a.least = 2;
    CUtensorMap tk, tv;
    if (!attention_maps(kv, TILE, &tk, &tv)) return cudaErrorInvalidValue;
    const int64_t units = (int64_t)kv.heads * ((int64_t)a.p.m * a.group / ROWS + std::min(kv.seqs, a.p.m)) + TARGET;    // at most
    const unsigned grid = (unsigned)std::min<int64_t>(units, dev.num_sms);
    return with_type(kv.type, [&](auto x) -> cudaError_t {
        using T = decltype(x);
        if constexpr (sizeof(T) == 4) {
            return cudaErrorInvalidValue;
        } else {
            auto go = [&](auto d) -> cudaError_t {
                constexpr int D = decltype(d)::value;
                constexpr size_t smem = Cfg<D>::STAGES_END + sizeof(Shared);
                static_assert(smem <= 227 * 1024, "shared memory");
                cudaError_t e = set_kernel_smem<attention_chunk_kernel<T, D>>(dev.device, smem);
                if (e != cudaSuccess) return e;
                e = launch_dependent(attention_chunk_kernel<T, D>, dim3(grid), THREADS, smem, stream, tk, tv, a);
                return e == cudaSuccess ? launch_attention_join(dev, a, D, ROWS, stream) : e;
            };
            return kv.dim == 64 ? go(std::integral_constant<int, 64>{}) : go(std::integral_constant<int, 128>{});
        }
    });
}

}  // namespace q8
