// gemm_mxfp4.cu -- the product of two MXFP4 matrices on the block-scaled tensor cores:
//   y[t][r] = sum_b 2^(Ew[r][b] + Ex[t][b]) sum_{i<32} w[r][32b+i] x[t][32b+i],  f32 accumulation.
//
// The weights are the MMA's A operand for every m (128 weight rows = 128 TMEM lanes), the tokens
// its N columns: a few tokens cost a narrow MMA, never a padded 128-row one, and the epilogue's
// lanes hold consecutive outputs of a token, so its stores are contiguous as they come.
//
// Tile: 128 weight rows x BN tokens, k in steps of 256 values (a 128-byte row of codes, 8 scales).
// Warp roles (192 threads):
//   warps 0-3   epilogue: tensor memory -> y, each warp its 32 lanes (warp index = lane quarter)
//   warp 4      producer: TMA of both code tiles (128-byte swizzle), bulk copies of the scale tiles
//   warp 5      tensor memory allocator and MMA issuer: per step the scale tiles go to tensor
//               memory as they are stored (tcgen05.cp), then four K = 64 MMAs
// Two accumulators in tensor memory: a tile's epilogue overlaps the next tile's MMAs.
//
// Few tokens: narrow stages, so two CTAs fit an SM where there are more row tiles than SMs.
// Few output tiles: the CTAs of a cluster split a tile's k among them.  Each sends its
// partial sums to the cluster's shared memories (rank c owns BN / CL of the tile's columns), and
// the owner adds them in rank order, so the result does not depend on timing.
//
// What bounds it: the weight stream for few tokens (5 x 64448 x 4096: 24.4 us for 142 MB with the
// activation's quantization, 0.86 of the copy rate; 1 x 4096 x 4096, 32 tiles shared by four CTAs each:
// 5.4 us with weights from HBM, latency), the MMAs for many (pairs of CTAs, below: 4095 x 20480 x 8192 with
// its quantizer 207 us in a burst, 6.6 PFLOP/s, and 227-235 call after call, 5.9, at the clock that the power
// limit then leaves).
// No rounding between the codes and y: products of codes and scales are exact, sums are the tensor
// cores' f32, y is rounded once.
#include "launch.h"
#include "mxfp4.cuh"
#include "tcgen05.cuh"
#include "types.cuh"

namespace q8 {
namespace {

constexpr int BM = 128;
constexpr int BK = 256;                    // values per k step
constexpr int ROW_BYTES = BK / 2;
constexpr int A_BYTES = BM * ROW_BYTES;
constexpr int SC_BYTES = BK / MX_TILE_K * MX_TILE_BYTES;   // a 128-row scale tile of one step
constexpr int THREADS = 192;
constexpr int SMEM_MAX = 232448;

// XSTEPS > 0: the CTA quantizes the activation itself and keeps its part of k (at most XSTEPS steps)
// in shared memory for all of its tiles; the stages then hold weights alone.
// PER_SM = 2: two CTAs to an SM, which do not share tiles.
template <int BN_, int STAGES_, int XSTEPS_ = 0, int PER_SM_ = 1>
struct Cfg {
    static constexpr int PER_SM = PER_SM_;
    static constexpr int BN = BN_;
    static constexpr int STAGES = STAGES_;
    static constexpr int XSTEPS = XSTEPS_;
    static constexpr int XSLOTS = XSTEPS > 0 ? XSTEPS : STAGES;
    static constexpr int NSB = BN > 128 ? 2 : 1;             // scale tiles that BN tokens touch
    static constexpr int B_BYTES = BN * ROW_BYTES;
    static constexpr bool SPLIT = BN <= 128 && PER_SM == 1;  // room for the cluster's partial sums
    static constexpr int OFF_A = 0;
    static constexpr int OFF_B = OFF_A + STAGES * A_BYTES;
    static constexpr int OFF_SA = OFF_B + XSLOTS * B_BYTES;
    static constexpr int OFF_SB = OFF_SA + STAGES * SC_BYTES;
    static constexpr int OFF_RED = OFF_SB + XSLOTS * NSB * SC_BYTES;
    static constexpr int OFF_BAR = OFF_RED + (SPLIT ? (BN < 32 ? 32 : BN) * BM * 4 : 0);   // 4 columns a rank at least
    static constexpr int OFF_MISC = OFF_BAR + (2 * STAGES + 4 + 4) * 8;
    static constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;   // + slack for 1024-byte base alignment
    // Tensor memory: two accumulators, then two slots of scales (weights 8 columns, tokens 8 per
    // scale tile), so that a step's copies do not wait for the previous step's MMAs.
    static constexpr int SC_COLS = 8 + 8 * NSB;
    static constexpr int COL_SC = 2 * BN;
    static constexpr int NEED = COL_SC + 2 * SC_COLS;
    static constexpr int TMEM_COLS = NEED <= 64 ? 64 : NEED <= 128 ? 128 : NEED <= 256 ? 256 : 512;
    static_assert(TMEM_COLS * PER_SM <= 512 && (SMEM_BYTES + 1024) * PER_SM <= SMEM_MAX + 1024, "capacity");
    // Instruction descriptor, block-scaled: B scale byte pair (bits 4-5), A and B e2m1 (bits 7-9,
    // 10-11 = 1), N >> 3 (17-22), scales e8m0 (23), M >> 4 (24-28), A scale byte pair (29-30).
    static constexpr uint32_t IDESC = (1u << 7) | (1u << 10) | ((uint32_t)(BN >> 3) << 17) | (1u << 23) |
                                      ((uint32_t)(BM >> 4) << 24);
};

// Descriptor of a scale tile's part: 32 rows of 16 bytes, 8-row groups 128 bytes apart, no swizzle.
__device__ __forceinline__ uint64_t smem_desc_scales(uint32_t saddr)
{
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)1 << 16) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
}

// 32 rows x 128 bits to 4 columns of tensor memory, repeated in each warp's 32 lanes.
__device__ __forceinline__ void tc_copy_scales(uint32_t taddr, uint64_t sdesc)
{
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}

__device__ __forceinline__ void tc_mma_mxf4(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                            uint32_t sa_tmem, uint32_t sb_tmem, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
        ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sa_tmem), "r"(sb_tmem), "r"(accumulate)
        : "memory");
}

// 32 lanes (this warp's) x 16 columns: thread = lane, register = column.
__device__ __forceinline__ void tc_ld_x16(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// 32 lanes x 32 columns, asynchronous: the registers are valid after tc_wait_ld.
__device__ __forceinline__ void tc_ld_x32(uint32_t taddr, uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,"
        "%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}
// Waits for this thread's loads from tensor memory; binds the registers to the wait.
template <int N>
__device__ __forceinline__ void tc_wait_ld(uint32_t (&a)[N][32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < 32; ++j) asm volatile("" : "+r"(a[i][j]));
}

// 32 lanes x N columns.
__device__ __forceinline__ void tc_columns(uint32_t taddr, uint32_t (&v)[1][16]) { tc_ld_x16(taddr, v[0]); }
template <int N>
__device__ __forceinline__ void tc_columns(uint32_t taddr, uint32_t (&v)[N][32])
{
#pragma unroll
    for (int i = 0; i < N; ++i) tc_ld_x32(taddr + 32 * i, v[i]);
    tc_wait_ld(v);
}

// ---- clusters ----
__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync_all()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_addr(uint32_t saddr, uint32_t rank)
{
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
    return r;
}
__device__ __forceinline__ void cluster_store4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void cluster_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// wait_or_abort whose success also orders what other CTAs of the cluster did before arriving: the
// completed phase is read once more with the cluster's scope (a fence would wait for this thread's
// own stores to the other CTAs too).
__device__ __forceinline__ bool wait_cluster(uint64_t *bar, uint32_t parity, int *status, volatile int *abort_flag)
{
    if (!wait_or_abort(bar, parity, status, abort_flag)) return false;
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
    return ok != 0;
}

struct Work {
    int m, n;
    int steps;        // k / BK
    int tiles;        // output tiles: token tile fastest
    int token_tiles;
    int first_wait;   // 1: the weights too may come from the kernel before this one
};

// X: the activation's type where the CTA quantizes it (xf, rows ldx elements apart), else unused.
template <typename C, typename T, typename X>
__global__ void __launch_bounds__(THREADS, C::PER_SM)
    gemm_mxfp4_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                      const uint8_t *__restrict__ wsc, const uint8_t *__restrict__ xsc, const X *__restrict__ xf,
                      int64_t ldx, T *__restrict__ y, Work wk, int CL, int *status)
{
    constexpr bool OWN_X = C::XSTEPS > 0;
    constexpr int BN = C::BN, STAGES = C::STAGES, NSB = C::NSB, B_BYTES = C::B_BYTES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
    uint64_t *empty = full + STAGES, *acc_full = empty + STAGES, *acc_empty = acc_full + 2;
    uint64_t *red_full = acc_empty + 2, *red_empty = red_full + 1, *drained = red_empty + 1, *x_ready = drained + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::OFF_MISC + 4);

    // Warp-uniform to the compiler too: the roles' loops then live in uniform registers.
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const bool shared = C::SPLIT && CL > 1;                   // a tile's k, by a cluster
    const uint32_t rank = shared ? cluster_rank() : 0;
    const int cluster = blockIdx.x / CL, clusters = gridDim.x / CL;
    const int ks0 = wk.steps * (int)rank / CL, ks1 = wk.steps * ((int)rank + 1) / CL;
    const int ktiles = wk.steps * (BK / MX_TILE_K);

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
        for (int s = 0; s < 2; ++s) { mbar_init(&acc_full[s], 1); mbar_init(&acc_empty[s], 4); }
        mbar_init(red_full, 4 * CL);
        mbar_init(red_empty, 4 * CL);
        mbar_init(drained, 1);
        mbar_init(x_ready, 4);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 5) tc_alloc(tmem_slot, C::TMEM_COLS);
    if (warp == 4 && lane == 0) {
        prefetch_tensormap(&tm_w);
        if (!OWN_X) prefetch_tensormap(&tm_x);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // Every rank's barriers exist before anyone arrives on them: the epilogue waits for it, the others
    // when they are done.
    if (shared) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);

    if (warp == 4) {
        // ------------------------------ producer ------------------------------
        // Everything that a tile fixes is computed once per tile: this thread's issue latency
        // paces the pipeline, and a division costs as much as several of its copies.
        const int last_sb = (wk.m + MX_TILE_ROWS - 1) / MX_TILE_ROWS;    // scale tiles of the tokens
        const int64_t sc_tile = (int64_t)ktiles * MX_TILE_BYTES;         // bytes of 128 rows' scales
        int row0, tok0, nsb;
        const uint8_t *wsp, *xsp;
        uint32_t bytes;
        auto enter = [&](int tile) {
            const int rt = tile / wk.token_tiles, tt = tile - rt * wk.token_tiles;
            const int sb0 = tt * BN / MX_TILE_ROWS;
            row0 = rt * BM;
            tok0 = tt * BN;
            nsb = min(NSB, last_sb - sb0);
            wsp = wsc + rt * sc_tile + ks0 * SC_BYTES;
            xsp = xsc + sb0 * sc_tile + ks0 * SC_BYTES;
            bytes = A_BYTES + SC_BYTES + (OWN_X ? 0 : B_BYTES + SC_BYTES * nsb);
        };
        auto load_w = [&](int st, int ks) {
            mbar_arrive_expect_tx(&full[st], bytes);
            tma_load_2d(smem + C::OFF_A + st * A_BYTES, &tm_w, ks * ROW_BYTES, row0, &full[st]);
            bulk_g2s(smem + C::OFF_SA + st * SC_BYTES, wsp, SC_BYTES, &full[st]);
        };
        auto load_x = [&](int st, int ks) {
            tma_load_2d(smem + C::OFF_B + st * B_BYTES, &tm_x, ks * ROW_BYTES, tok0, &full[st]);
            bulk_g2s(smem + C::OFF_SB + st * NSB * SC_BYTES, xsp, SC_BYTES, &full[st]);
            if (NSB > 1 && nsb > 1) bulk_g2s(smem + C::OFF_SB + (st * NSB + 1) * SC_BYTES, xsp + sc_tile, SC_BYTES, &full[st]);
        };
        // The first stages' weights before the wait for the previous kernel, which in a fused
        // call is the activation's quantizer and does not write them.
        if (wk.first_wait) griddep_wait();
        int early = 0;
        for (int tile = cluster; tile < wk.tiles && early < STAGES; tile += clusters) {
            enter(tile);
            for (int ks = ks0; ks < ks1 && early < STAGES; ++ks, ++early) {
                if (elect_one()) load_w(early, ks);
                wsp += SC_BYTES;
            }
        }
        if (!wk.first_wait) griddep_wait();
        griddep_launch_dependents();
        int it = 0, st = 0;
        uint32_t phase = 1;
        bool ok = true;
        for (int tile = cluster; ok && tile < wk.tiles; tile += clusters) {
            enter(tile);
            for (int ks = ks0; ks < ks1; ++ks, ++it) {
                if (it >= early) {
                    ok = __all_sync(0xffffffffu, wait_or_abort(&empty[st], phase, status, abort_flag));
                    if (!ok) break;
                }
                if (elect_one()) {
                    if (it >= early) load_w(st, ks);
                    if (!OWN_X) load_x(st, ks);
                }
                wsp += SC_BYTES;
                xsp += SC_BYTES;
                if (++st == STAGES) {
                    st = 0;
                    phase ^= 1;
                }
            }
        }
        // Never leave with a copy into this CTA's shared memory in flight.
        for (int i = it > STAGES ? it - STAGES : 0; i < it; ++i)
            mbar_wait_drain(&full[i % STAGES], (i / STAGES) & 1, status);
    } else if (warp == 5) {
        // ------------------------------ MMA issuer ------------------------------
        // Every role waits for the previous kernel first: a pipeline wait's time limit is for this kernel's
        // own copies and MMAs, not for what is left of that one.
        griddep_wait();
        const uint64_t adesc0 = smem_desc_sw128(smem_u32(smem + C::OFF_A));
        const uint64_t bdesc0 = smem_desc_sw128(smem_u32(smem + C::OFF_B));
        const uint64_t sadesc0 = smem_desc_scales(smem_u32(smem + C::OFF_SA));
        const uint64_t sbdesc0 = smem_desc_scales(smem_u32(smem + C::OFF_SB));
        // Steps go in pairs where the second one's data is there: the tensor pipe runs copies and
        // MMAs in order and pays for each change between them.
        auto copy_scales = [&](int slot, int st, int ks) {
            const int xs = OWN_X ? ks - ks0 : st;     // where the tokens' operand is
            const uint32_t sa = tmem + C::COL_SC + slot * C::SC_COLS, sb = sa + 8;
#pragma unroll
            for (int g = 0; g < 2; ++g) {        // the step's two groups of 128 values
                tc_copy_scales(sa + 4 * g, sadesc0 + (uint64_t)((st * SC_BYTES + g * MX_TILE_BYTES) >> 4));
#pragma unroll
                for (int b = 0; b < NSB; ++b)
                    tc_copy_scales(sb + 4 * (NSB * g + b),
                                   sbdesc0 + (uint64_t)(((xs * NSB + b) * SC_BYTES + g * MX_TILE_BYTES) >> 4));
            }
        };
        auto multiply = [&](int slot, int st, int ks, uint32_t d_tmem, uint32_t sb_shift) {
            const int xs = OWN_X ? ks - ks0 : st;
            const bool first = ks == ks0;
            const uint32_t sa = tmem + C::COL_SC + slot * C::SC_COLS, sb = sa + 8 + sb_shift;
            const uint64_t ad = adesc0 + (uint64_t)(st * (A_BYTES >> 4));
            const uint64_t bd = bdesc0 + (uint64_t)(xs * (B_BYTES >> 4));
#pragma unroll
            for (int j = 0; j < 4; ++j) {        // 64 values: bytes 2 (j % 2) and next of each scale word
                const uint32_t id = C::IDESC | ((uint32_t)(2 * (j & 1)) << 4) | ((uint32_t)(2 * (j & 1)) << 29);
                tc_mma_mxf4(d_tmem, ad + 2 * j, bd + 2 * j, id, sa + 4 * (j >> 1), sb + 4 * NSB * (j >> 1), !first || j > 0);
            }
            tc_commit(&empty[st]);
        };
        int st = 0, i = 0;
        uint32_t phase = 0;
        bool ok = !OWN_X || __all_sync(0xffffffffu, wait_or_abort(x_ready, 0, status, abort_flag));
        for (int tile = cluster; ok && tile < wk.tiles; tile += clusters, ++i) {
            const int acc = i & 1;
            ok = __all_sync(0xffffffffu, wait_or_abort(&acc_empty[acc], ((i >> 1) & 1) ^ 1, status, abort_flag));
            if (!ok) break;
            // the first of the tile's tokens within its 128-row scale tile: a column for each 32
            const uint32_t sb_shift = (uint32_t)(tile % wk.token_tiles * BN % MX_TILE_ROWS / 32);
            for (int ks = ks0; ks < ks1;) {
                ok = __all_sync(0xffffffffu, wait_or_abort(&full[st], phase, status, abort_flag));
                if (!ok) break;
                const int st1 = st + 1 == STAGES ? 0 : st + 1;
                const bool two = ks + 1 < ks1 &&
                                 __all_sync(0xffffffffu, mbar_try_wait(&full[st1], st1 == 0 ? phase ^ 1 : phase));
                tc_fence_after();
                if (elect_one()) {
                    copy_scales(0, st, ks);
                    if (two) copy_scales(1, st1, ks + 1);
                    multiply(0, st, ks, tmem + acc * BN, sb_shift);
                    if (two) multiply(1, st1, ks + 1, tmem + acc * BN, sb_shift);
                    if (ks + (two ? 2 : 1) == ks1) tc_commit(&acc_full[acc]);
                }
                for (int n = two ? 2 : 1; n; --n, ++ks)
                    if (++st == STAGES) {
                        st = 0;
                        phase ^= 1;
                    }
            }
        }
        // Tensor memory is not freed under an MMA: a last commit arrives after all of them.
        if (elect_one()) tc_commit(drained);
        mbar_wait_drain(drained, 0, status);
    } else {
        // ------------------------------ epilogue ------------------------------
        const uint32_t lane_base = (uint32_t)(32 * warp) << 16;
        const int row = 32 * warp + lane;
        float *red = reinterpret_cast<float *>(smem + C::OFF_RED);
        griddep_wait();
        if constexpr (OWN_X) {
            // First the activation: a warp has 256 values of a token at a time, and writes them as
            // the TMA would have (token rows of 128 bytes, 16-byte units swizzled by the row).
            const int tasks = wk.m * (ks1 - ks0);
            constexpr int DEPTH = 4;                  // loads under way
            for (int task0 = warp; task0 < tasks; task0 += 4 * DEPTH) {
                uint4 in[DEPTH][sizeof(X) / 2];
#pragma unroll
                for (int d = 0; d < DEPTH; ++d) {
                    const int task = task0 + 4 * d, t = task % wk.m, s = task / wk.m;
                    const uint4 *src = reinterpret_cast<const uint4 *>(xf + t * ldx + (int64_t)(ks0 + s) * BK + lane * 8);
#pragma unroll
                    for (int h = 0; h < (int)sizeof(X) / 2; ++h) in[d][h] = task < tasks ? src[h] : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int d = 0; d < DEPTH; ++d) {
                    const int task = task0 + 4 * d, t = task % wk.m, s = task / wk.m;
                    if (task >= tasks) break;
                    const MxChunk q = mx_quantize8<X>(in[d]);
                    uint8_t *dst = smem + C::OFF_B + s * B_BYTES + t * ROW_BYTES + (((lane >> 2) ^ (t & 7)) << 4) + (lane & 3) * 4;
                    *reinterpret_cast<uint32_t *>(dst) = q.codes;
                    if ((lane & 15) == 0)
                        *reinterpret_cast<uint32_t *>(smem + C::OFF_SB + s * SC_BYTES + (lane >> 4) * MX_TILE_BYTES + t * 16) = q.scales;
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(x_ready);
        }
        int i = 0;
        bool met = false;                      // the cluster's first barrier has been waited for
        for (int tile = cluster; tile < wk.tiles; tile += clusters, ++i) {
            const int acc = i & 1;
            const int64_t r = (int64_t)(tile / wk.token_tiles) * BM + row;
            const int tok0 = tile % wk.token_tiles * BN;
            const int cols = min(BN, wk.m - tok0);
            if (!__all_sync(0xffffffffu, wait_or_abort(&acc_full[acc], (i >> 1) & 1, status, abort_flag))) break;
            tc_fence_after();
            T *dst = y + (int64_t)tok0 * wk.n + r;
            // columns read from tensor memory at once
            constexpr int LD = BN < 32 ? BN : 32, LDS = BN < 64 ? 1 : 2, PART = LD * LDS;
            if (!shared) {
#pragma unroll 1
                for (int c0 = 0; c0 < cols; c0 += PART) {
                    uint32_t v[LDS][LD];
                    tc_columns(tmem + lane_base + acc * BN + c0, v);
                    if (r >= wk.n) continue;
                    if (c0 + PART <= cols) {
#pragma unroll
                        for (int c = 0; c < PART; ++c, dst += wk.n) *dst = from_f32<T>(__uint_as_float(v[c / LD][c % LD]));
                    } else {
#pragma unroll
                        for (int c = 0; c < PART; ++c, dst += wk.n)
                            if (c0 + c < cols) *dst = from_f32<T>(__uint_as_float(v[c / LD][c % LD]));
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&acc_empty[acc]);
            } else if constexpr (C::SPLIT) {
                // BN and CL are powers of two: rank o owns the columns of BN / CL / 4 groups of four (at
                // least one) from its first on; its partial sums stand as [rank][group][row][four].
                const int groups = BN / 4 / CL > 0 ? BN / 4 / CL : 1, shift = 31 - __clz(groups);
                if (!met) {
                    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
                    met = true;
                } else if (!__all_sync(0xffffffffu, wait_cluster(red_empty, (i & 1) ^ 1, status, abort_flag))) {
                    break;
                }
                const uint32_t mine = smem_u32(red + ((int)rank * groups * BM + row) * 4);
#pragma unroll 1
                for (int c0 = 0; c0 < cols; c0 += PART) {
                    uint32_t v[LDS][LD];
                    tc_columns(tmem + lane_base + acc * BN + c0, v);
#pragma unroll
                    for (int c = 0; c < PART; c += 4) {
                        const int g = (c0 + c) >> 2;
                        if (c0 + c < cols)
                            cluster_store4(cluster_addr(mine + (uint32_t)((g & (groups - 1)) * BM * 16), g >> shift),
                                           v[c / LD][c % LD], v[c / LD][c % LD + 1], v[c / LD][c % LD + 2],
                                           v[c / LD][c % LD + 3]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&acc_empty[acc]);
                if (lane < CL) cluster_arrive(cluster_addr(smem_u32(red_full), lane));
                if (!__all_sync(0xffffffffu, wait_cluster(red_full, i & 1, status, abort_flag))) break;
                const int own0 = (int)rank * groups * 4;
                const float4 *parts = reinterpret_cast<const float4 *>(red) + row;
#pragma unroll 1
                for (int g = 0; g < groups && own0 + 4 * g < cols; ++g) {
                    float4 part[8];
#pragma unroll
                    for (int src = 0; src < 8; ++src)
                        part[src] = src < CL ? parts[(src * groups + g) * BM] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    float sum[4] = {part[0].x, part[0].y, part[0].z, part[0].w};
#pragma unroll
                    for (int src = 1; src < 8; ++src)
                        if (src < CL) {                                          // in rank order
                            sum[0] += part[src].x;
                            sum[1] += part[src].y;
                            sum[2] += part[src].z;
                            sum[3] += part[src].w;
                        }
                    if (r < wk.n)
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            if (own0 + 4 * g + c < cols) dst[(int64_t)(own0 + 4 * g + c) * wk.n] = from_f32<T>(sum[c]);
                }
                __syncwarp();
                if (lane < CL) cluster_arrive(cluster_addr(smem_u32(red_empty), lane));
            }
        }
        if (shared && !met) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }

    __syncwarp();
    if (shared && warp >= 4) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    tc_fence_before();
    __syncthreads();
    if (shared) cluster_sync_all();         // nobody leaves while others may still write to it
    if (warp == 5) {
        tc_fence_after();
        tc_dealloc(tmem, C::TMEM_COLS);
    }
}

// Clusters of CL CTAs that are resident at once (looked up once per device, kernel and CL).
template <typename C, typename T, typename X>
cudaError_t resident_clusters(const DeviceInfo &dev, int CL, int *count)
{
    static std::atomic<int> known[kAttrDevices][4];
    const int slot = CL == 1 ? 0 : CL == 2 ? 1 : CL == 4 ? 2 : 3;
    const bool cache = dev.device >= 0 && dev.device < kAttrDevices;
    if (CL == 1) {
        *count = dev.num_sms * C::PER_SM;
        return cudaSuccess;
    }
    if (cache && (*count = known[dev.device][slot].load(std::memory_order_relaxed)) > 0) return cudaSuccess;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(dev.num_sms / CL * CL));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)CL;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int got = 0;
    cudaError_t e = cudaOccupancyMaxActiveClusters(&got, gemm_mxfp4_kernel<C, T, X>, &cfg);
    if (e != cudaSuccess) return e;
    *count = got < dev.num_sms / CL ? got : dev.num_sms / CL;
    if (*count < 1) return cudaErrorInvalidConfiguration;
    if (cache) known[dev.device][slot].store(*count, std::memory_order_relaxed);
    return cudaSuccess;
}

// x, xsc: the quantized activation (C::XSTEPS = 0); else xf, ldx: the activation itself.
template <typename C, typename T, typename X>
cudaError_t launch_tiles(const DeviceInfo &dev, const uint8_t *w, const uint8_t *wsc, const uint8_t *x,
                         const uint8_t *xsc, const X *xf, int64_t ldx, T *y, int64_t m, int64_t n, int64_t k, int CL,
                         bool pdl, cudaStream_t stream)
{
    cudaError_t e = set_kernel_smem<gemm_mxfp4_kernel<C, T, X>>(dev.device, C::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    int resident = 0;
    if ((e = resident_clusters<C, T, X>(dev, CL, &resident)) != cudaSuccess) return e;
    CUtensorMap tm_w, tm_x;
    if (!encode_2d(&tm_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, w, (uint64_t)k / 2, (uint64_t)n, (uint64_t)k / 2, ROW_BYTES, BM,
                   CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    if (C::XSTEPS > 0)
        tm_x = tm_w;                                   // unused
    else if (!encode_2d(&tm_x, CU_TENSOR_MAP_DATA_TYPE_UINT8, x, (uint64_t)k / 2, (uint64_t)m, (uint64_t)k / 2, ROW_BYTES,
                        C::BN, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    Work wk;
    wk.m = (int)m;
    wk.n = (int)n;
    wk.steps = (int)(k / BK);
    wk.token_tiles = (int)((m + C::BN - 1) / C::BN);
    const int64_t tiles = (n + BM - 1) / BM * wk.token_tiles;
    if (tiles > INT32_MAX / 2) return cudaErrorInvalidValue;
    wk.tiles = (int)tiles;
    wk.first_wait = pdl ? 0 : 1;
    const int64_t clusters = tiles < resident ? tiles : resident;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(clusters * CL));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)CL;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CL > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, gemm_mxfp4_kernel<C, T, X>, tm_w, tm_x, wsc, xsc, xf, ldx, y, wk, CL, dev.status);
}

// ---------------------------------------------------------------------------------------
// Many tokens: a pair of CTAs (two SMs) on one tile of 256 weight rows x 256 or 192 tokens.
//
// What bounds one CTA's MMAs is reading their operands from shared memory: at 64 values of k,
// 128 x N takes (128 + N) * 32 bytes, and the measured times (126, 151, 180 cycles for N = 128,
// 192, 256) are 64 bytes a cycle.  A pair's MMA (cta_group::2) leaves half of the tokens' operand to
// each SM: 8 KB for 128 x 256 outputs an SM, which is what its arithmetic takes (128 cycles).
//
// Each CTA loads its 128 weight rows, its half of the tokens, its rows' scales and all tokens' scales;
// all copies of a stage arrive on the first CTA's barrier, whose issuer runs the MMAs of both, each
// SM keeping its 128 rows' results.  Eight epilogue warps take an accumulator into registers at once
// (half of the columns each), release it, then store.  256 tokens: two accumulators would leave tensor
// memory no room for the scales, so the next tile's MMAs wait for the hand-over (2.4 us a tile).  192
// tokens: two, and no such wait, for 112 cycles of operands where the arithmetic takes 96.  So 192 is
// faster up to k = 4096 (2048 x 12288 x 4096: 35.0 us, 41.0 by 256; call after call 37.4 and 40.9) and about
// equal at 8192 (4095 x 20480: 187.5 and 190.8; call after call 214 and 212).
//
// Tiles that do not fill a last round of all pairs are cut into parts of 128 or 64 tokens, so that
// the round takes less: a part's MMA reads 4 KB of its 128 weight rows whatever its tokens are (5 KB with
// 64 of 256 tokens, 8 with all), so a quarter costs 0.6 of a tile, not 0.25.
// ---------------------------------------------------------------------------------------
template <int BN_>
struct PairCfg {
    static constexpr int BN = BN_, ACCS = BN < 256 ? 2 : 1, STAGES = BN < 256 ? 7 : 6;
    static constexpr int NSB = 2;                            // scale tiles that BN tokens touch
    static constexpr int B_BYTES = BN / 2 * ROW_BYTES, SB_BYTES = NSB * SC_BYTES;
    static constexpr int OFF_A = 0;
    static constexpr int OFF_B = OFF_A + STAGES * A_BYTES;
    static constexpr int OFF_SA = OFF_B + STAGES * B_BYTES;
    static constexpr int OFF_SB = OFF_SA + STAGES * SC_BYTES;
    static constexpr int OFF_BAR = OFF_SB + STAGES * SB_BYTES;
    static constexpr int OFF_MISC = OFF_BAR + (2 * STAGES + 2 * ACCS + 1) * 8;
    static constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;
    static constexpr int EPI_WARPS = 8, THREADS = (EPI_WARPS + 2) * 32;
    static constexpr int COL_SC = ACCS * BN, SC_COLS = 8 + 8 * NSB, TMEM_COLS = 512;
    static constexpr uint32_t IDESC = (1u << 7) | (1u << 10) | (1u << 23) | ((uint32_t)(2 * BM >> 4) << 24);  // without N
    static_assert(SMEM_BYTES <= SMEM_MAX && COL_SC + 2 * SC_COLS <= TMEM_COLS && B_BYTES % 1024 == 0, "capacity");
    // A tile's or part's first column of scales must be even (an MMA cannot start at an odd one), and
    // its scales within two 128-row tiles.
    static_assert(BN % 64 == 0 && (BN == 192 || BN == 256), "whole pairs of scale columns");
};

__device__ __forceinline__ void pair_copy_scales(uint32_t taddr, uint64_t sdesc)
{
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}
__device__ __forceinline__ void pair_mma(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t sa_tmem, uint32_t sb_tmem, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
        ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sa_tmem), "r"(sb_tmem), "r"(accumulate)
        : "memory");
}
// Arrives on both CTAs' barrier of that place once the MMAs issued before have completed.
__device__ __forceinline__ void pair_commit(uint64_t *bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
        ::"r"(smem_u32(bar)), "h"((uint16_t)3)
        : "memory");
}
// A TMA load into this CTA's shared memory that completes on a barrier of the pair's first CTA.
__device__ __forceinline__ void pair_load_2d(void *dst, const CUtensorMap *map, int32_t x, int32_t y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];"
        ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// Units of work: whole tiles (token tile fastest), then the cut ones' parts.
struct PairWork {
    int m, n;
    int steps;        // k / BK
    int token_tiles;
    int whole;        // tiles that stay whole: a multiple of the pairs, or all
    int parts;        // the others are cut into so many
    int units;
    int first_wait;   // as Work's
};

struct PairUnit {
    int row, tok, tokens;     // row tile of 256, first token, tokens
};
template <int BN>
__device__ __forceinline__ PairUnit pair_unit(const PairWork &wk, int u)
{
    const bool cut = u >= wk.whole;
    const int part = u - wk.whole, above = cut ? part / wk.parts : 0;
    const int tile = cut ? wk.whole + above : u;
    PairUnit r;
    r.row = tile / wk.token_tiles;
    r.tokens = cut ? BN / wk.parts : BN;
    r.tok = (tile - r.row * wk.token_tiles) * BN + (cut ? part - above * wk.parts : 0) * r.tokens;
    return r;
}

// tm_xp: the tokens of a part (its box has fewer rows than tm_x's).
template <typename C, typename T>
__global__ void __launch_bounds__(C::THREADS, 1)
    gemm_mxfp4_pair_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                           const __grid_constant__ CUtensorMap tm_xp, const __grid_constant__ CUtensorMap tm_ws,
                           const __grid_constant__ CUtensorMap tm_xs, T *__restrict__ y, PairWork wk, int *status)
{
    constexpr int STAGES = C::STAGES, ACCS = C::ACCS, NSB = C::NSB;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);        // used in the first CTA
    uint64_t *empty = full + STAGES, *acc_full = empty + STAGES, *acc_empty = acc_full + ACCS, *drained = acc_empty + ACCS;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::OFF_MISC + 4);

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
        for (int s = 0; s < ACCS; ++s) { mbar_init(&acc_full[s], 1); mbar_init(&acc_empty[s], 2 * C::EPI_WARPS); }
        mbar_init(drained, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == C::EPI_WARPS + 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(C::TMEM_COLS) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    if (warp == C::EPI_WARPS && lane == 0) {
        prefetch_tensormap(&tm_w);
        prefetch_tensormap(&tm_x);
        prefetch_tensormap(&tm_xp);
        prefetch_tensormap(&tm_ws);
        prefetch_tensormap(&tm_xs);
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);

    if (warp == C::EPI_WARPS) {
        // ------------------------------ producer ------------------------------
        int row_tile, tok, scale_row;
        uint32_t bytes;                                                 // both CTAs' of a stage
        const CUtensorMap *map_x;
        auto enter = [&](int u) {
            const PairUnit unit = pair_unit<C::BN>(wk, u);
            row_tile = 2 * unit.row + (int)rank;                        // this CTA's 128 rows
            tok = unit.tok + (int)rank * (unit.tokens / 2);             // and its half of the tokens
            scale_row = unit.tok / MX_TILE_ROWS;
            map_x = u < wk.whole ? &tm_x : &tm_xp;
            bytes = 2 * (A_BYTES + SC_BYTES + C::SB_BYTES) + (uint32_t)unit.tokens * ROW_BYTES;
        };
        auto load_w = [&](int st, int ks) {
            const uint32_t bar = cluster_addr(smem_u32(&full[st]), 0);
            if (rank == 0) mbar_arrive_expect_tx(&full[st], bytes);
            pair_load_2d(smem + C::OFF_A + st * A_BYTES, &tm_w, ks * ROW_BYTES, row_tile * BM, bar);
            pair_load_2d(smem + C::OFF_SA + st * SC_BYTES, &tm_ws, ks * (SC_BYTES / 8), row_tile, bar);
        };
        auto load_x = [&](int st, int ks) {
            const uint32_t bar = cluster_addr(smem_u32(&full[st]), 0);
            pair_load_2d(smem + C::OFF_B + st * C::B_BYTES, map_x, ks * ROW_BYTES, tok, bar);
            pair_load_2d(smem + C::OFF_SB + st * C::SB_BYTES, &tm_xs, ks * (SC_BYTES / 8), scale_row, bar);
        };
        // As in gemm_mxfp4_kernel: the first stages' weights before the wait in a fused call.
        if (wk.first_wait) griddep_wait();
        int early = 0;
        for (int u = pair; u < wk.units && early < STAGES; u += pairs) {
            enter(u);
            for (int ks = 0; ks < wk.steps && early < STAGES; ++ks, ++early)
                if (elect_one()) load_w(early, ks);
        }
        if (!wk.first_wait) griddep_wait();
        griddep_launch_dependents();
        int st = 0, it = 0;
        uint32_t phase = 1;
        bool ok = true;
        for (int u = pair; ok && u < wk.units; u += pairs) {
            enter(u);
            for (int ks = 0; ks < wk.steps; ++ks, ++it) {
                if (it >= early) {
                    ok = __all_sync(0xffffffffu, wait_or_abort(&empty[st], phase, status, abort_flag));
                    if (!ok) break;
                }
                if (elect_one()) {
                    if (it >= early) load_w(st, ks);
                    load_x(st, ks);
                }
                if (++st == STAGES) {
                    st = 0;
                    phase ^= 1;
                }
            }
        }
        // Neither CTA leaves with a copy in flight: the first one's barriers count both CTAs' copies,
        // and the other waits for it at the cluster's last barrier.
        if (rank == 0)
            for (int i = it > STAGES ? it - STAGES : 0; i < it; ++i)
                mbar_wait_drain(&full[i % STAGES], (i / STAGES) & 1, status);
        // Nor does it leave before the first CTA's last commits have arrived on its barriers.
        for (int i = it > STAGES ? it - STAGES : 0; i < it; ++i)
            wait_or_abort(&empty[i % STAGES], (i / STAGES) & 1, status, abort_flag);
    } else if (warp == C::EPI_WARPS + 1) {
        // ------------------------------ MMA issuer (first CTA) ------------------------------
        if (rank == 0) {
            griddep_wait();                                             // as in gemm_mxfp4_kernel
            const uint64_t adesc0 = smem_desc_sw128(smem_u32(smem + C::OFF_A));
            const uint64_t bdesc0 = smem_desc_sw128(smem_u32(smem + C::OFF_B));
            const uint64_t sadesc0 = smem_desc_scales(smem_u32(smem + C::OFF_SA));
            const uint64_t sbdesc0 = smem_desc_scales(smem_u32(smem + C::OFF_SB));
            auto copy_scales = [&](int slot, int st) {
                const uint32_t sa = tmem + C::COL_SC + slot * C::SC_COLS, sb = sa + 8;
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    pair_copy_scales(sa + 4 * g, sadesc0 + (uint64_t)((st * SC_BYTES + g * MX_TILE_BYTES) >> 4));
#pragma unroll
                    for (int b = 0; b < NSB; ++b)
                        pair_copy_scales(sb + 4 * (NSB * g + b),
                                         sbdesc0 + (uint64_t)((st * C::SB_BYTES + b * SC_BYTES + g * MX_TILE_BYTES) >> 4));
                }
            };
            uint32_t idesc = 0, sb_shift = 0;      // of the unit: N; its first token's column of scales
            auto multiply = [&](int slot, int st, uint32_t d_tmem, bool first) {
                const uint32_t sa = tmem + C::COL_SC + slot * C::SC_COLS, sb = sa + 8 + sb_shift;
                const uint64_t ad = adesc0 + (uint64_t)(st * (A_BYTES >> 4));
                const uint64_t bd = bdesc0 + (uint64_t)(st * (C::B_BYTES >> 4));
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t id = idesc | ((uint32_t)(2 * (j & 1)) << 4) | ((uint32_t)(2 * (j & 1)) << 29);
                    pair_mma(d_tmem, ad + 2 * j, bd + 2 * j, id, sa + 4 * (j >> 1), sb + 4 * NSB * (j >> 1), !first || j > 0);
                }
                pair_commit(&empty[st]);
            };
            int st = 0, i = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int u = pair; ok && u < wk.units; u += pairs, ++i) {
                const PairUnit unit = pair_unit<C::BN>(wk, u);
                idesc = C::IDESC | ((uint32_t)(unit.tokens >> 3) << 17);
                sb_shift = (uint32_t)(unit.tok % MX_TILE_ROWS / 32);
                const int acc = i % ACCS;
                ok = __all_sync(0xffffffffu, wait_or_abort(&acc_empty[acc], (i / ACCS & 1) ^ 1, status, abort_flag));
                if (!ok) break;
                for (int ks = 0; ks < wk.steps;) {
                    ok = __all_sync(0xffffffffu, wait_or_abort(&full[st], phase, status, abort_flag));
                    if (!ok) break;
                    const int st1 = st + 1 == STAGES ? 0 : st + 1;
                    const bool two = ks + 1 < wk.steps &&
                                     __all_sync(0xffffffffu, mbar_try_wait(&full[st1], st1 == 0 ? phase ^ 1 : phase));
                    tc_fence_after();
                    if (elect_one()) {
                        copy_scales(0, st);
                        if (two) copy_scales(1, st1);
                        multiply(0, st, tmem + acc * C::BN, ks == 0);
                        if (two) multiply(1, st1, tmem + acc * C::BN, false);
                        if (ks + (two ? 2 : 1) == wk.steps) pair_commit(&acc_full[acc]);
                    }
                    for (int n = two ? 2 : 1; n; --n, ++ks)
                        if (++st == STAGES) {
                            st = 0;
                            phase ^= 1;
                        }
                }
            }
            // Tensor memory is not freed under an MMA: a last commit arrives after all of them.
            if (elect_one())
                asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                             ::"r"(smem_u32(drained)) : "memory");
            mbar_wait_drain(drained, 0, status);
        }
    } else {
        // ------------------------------ epilogue ------------------------------
        griddep_wait();
        const int quarter = warp & 3, half = warp >> 2;                  // 32 lanes, half of the columns
        int i = 0;
        for (int u = pair; u < wk.units; u += pairs, ++i) {
            const PairUnit unit = pair_unit<C::BN>(wk, u);
            const int64_t r = (int64_t)(2 * unit.row + (int)rank) * BM + 32 * quarter + lane;
            const int per = unit.tokens / 2, tok0 = unit.tok + half * per;
            const int cols = min(per, wk.m - tok0);
            const int acc = i % ACCS;
            if (!__all_sync(0xffffffffu, wait_or_abort(&acc_full[acc], i / ACCS & 1, status, abort_flag))) break;
            tc_fence_after();
            constexpr int HALF = C::BN / 2, NQ = HALF / 32;
            uint32_t v[NQ][32];
#pragma unroll
            for (int q = 0; q < NQ; ++q)
                if (32 * q < per)
                    tc_ld_x32(tmem + ((uint32_t)(32 * quarter) << 16) + acc * C::BN + half * per + 32 * q, v[q]);
            tc_wait_ld(v);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) cluster_arrive(cluster_addr(smem_u32(&acc_empty[acc]), 0));
            if (r < wk.n) {
                T *dst = y + (int64_t)tok0 * wk.n + r;
                if (cols == HALF) {
#pragma unroll
                    for (int c = 0; c < HALF; ++c, dst += wk.n) *dst = from_f32<T>(__uint_as_float(v[c / 32][c % 32]));
                } else {
#pragma unroll
                    for (int c = 0; c < HALF; ++c, dst += wk.n)
                        if (c < cols) *dst = from_f32<T>(__uint_as_float(v[c / 32][c % 32]));
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    if (warp == C::EPI_WARPS + 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::TMEM_COLS) : "memory");
    }
}

// Into how many parts the tiles of a last round that leaves pairs idle are cut: as many as the pairs
// can take at once, down to 64 tokens (whole pairs of scale columns).
int pair_parts(int bn, int64_t tiles, int64_t pairs)
{
    const int64_t left = tiles % pairs;
    if (bn == 192) return left * 3 <= pairs ? 3 : 1;
    return left * 4 <= pairs ? 4 : left * 2 <= pairs ? 2 : 1;
}

template <typename C, typename T>
cudaError_t launch_pairs(const DeviceInfo &dev, const uint8_t *w, const uint8_t *wsc, const uint8_t *x,
                         const uint8_t *xsc, T *y, int64_t m, int64_t n, int64_t k, bool pdl, cudaStream_t stream)
{
    cudaError_t e = set_kernel_smem<gemm_mxfp4_pair_kernel<C, T>>(dev.device, C::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    const int64_t tiles = (n + 2 * BM - 1) / (2 * BM) * ((m + C::BN - 1) / C::BN);
    if (tiles > INT32_MAX / 2) return cudaErrorInvalidValue;
    const int64_t at_once = dev.num_sms / 2;
    PairWork wk{};
    wk.m = (int)m;
    wk.n = (int)n;
    wk.steps = (int)(k / BK);
    wk.token_tiles = (int)((m + C::BN - 1) / C::BN);
    wk.parts = pair_parts(C::BN, tiles, at_once);
    wk.whole = (int)(wk.parts > 1 ? tiles / at_once * at_once : tiles);
    wk.units = wk.whole + ((int)tiles - wk.whole) * wk.parts;
    wk.first_wait = pdl ? 0 : 1;
    const int64_t pairs = wk.units < at_once ? wk.units : at_once;
    const uint64_t sc_row = (uint64_t)k / MX_TILE_K * MX_TILE_BYTES;      // bytes of 128 rows' scales
    CUtensorMap tm_w, tm_x, tm_xp, tm_ws, tm_xs;
    if (!encode_2d(&tm_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, w, (uint64_t)k / 2, (uint64_t)n, (uint64_t)k / 2, ROW_BYTES, BM,
                   CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_2d(&tm_x, CU_TENSOR_MAP_DATA_TYPE_UINT8, x, (uint64_t)k / 2, (uint64_t)m, (uint64_t)k / 2, ROW_BYTES,
                   C::BN / 2, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_2d(&tm_xp, CU_TENSOR_MAP_DATA_TYPE_UINT8, x, (uint64_t)k / 2, (uint64_t)m, (uint64_t)k / 2, ROW_BYTES,
                   C::BN / 2 / wk.parts, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_2d(&tm_ws, CU_TENSOR_MAP_DATA_TYPE_UINT64, wsc, sc_row / 8, (uint64_t)(n + 127) / 128, sc_row,
                   SC_BYTES / 8, 1, CU_TENSOR_MAP_SWIZZLE_NONE) ||
        !encode_2d(&tm_xs, CU_TENSOR_MAP_DATA_TYPE_UINT64, xsc, sc_row / 8, (uint64_t)(m + 127) / 128, sc_row,
                   SC_BYTES / 8, C::NSB, CU_TENSOR_MAP_SWIZZLE_NONE))
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * pairs));
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, gemm_mxfp4_pair_kernel<C, T>, tm_w, tm_x, tm_xp, tm_ws, tm_xs, y, wk, dev.status);
}

}  // namespace

namespace {

// The tile shape of a product and how many CTAs share a tile's k: the least of
//   rounds * (steps of a CTA * time of a step + the tile's start and end + joining its partial sums)
// over the tile widths, the powers of two up to 8 that leave each CTA a step, and pairs (whose round
// takes no less than their epilogue's stores, and whose last round of cut tiles has its own times).
// The times, in ns, are fitted to every such choice measured at some 1000 sizes (m from 1 to 4095, n
// from 1000 to 64448, k from 512 to 20480, weights from HBM): what the formula takes is 0.4 % above the
// best choice on average, 21 % at worst (256 x 4096 x 4096: 6.7 us in 64-token tiles, 8.2 in 128-token
// ones, 10.8 if two share those, 8.3 by pairs; 1 x 2500 x 20480: 11.7 shared by four, 21.2 not shared;
// 4095 x 12288 x 4096: 64 by pairs with 192 tokens, 74 with 256, 80 in 192-token tiles of one CTA).
// Up to 16 tokens nothing of the choice depends on m, so that a token's sums are formed in the same order
// for every m, decoding and verifying: the join's cost is then that of all 16 columns whatever m is (against
// 6, at 40 sizes of the two choices: 7 % less on average at 1 token, 10 % at 15; 5073 x 2560 at 1 token 4.7 us
// not shared, 5.2 by two; 2282 x 2304 4.2 not shared, 4.05 by four).
GemmPlan plan_tiles(int sms, int64_t m, int64_t n, int64_t k)
{
    const int64_t rows = (n + BM - 1) / BM, steps = k / BK;
    // One token tile and more row tiles than SMs: two CTAs to an SM, so that the last tiles are read
    // beside others and not at the end by a few SMs (1, 8, 32 x 20480 x 4096: 160 tiles, 10.0, 9.9, 10.4 us;
    // 12.3, 12.6, 13.0 by one CTA to an SM; 8 x 64448 x 4096 25.0 and 27.0).
    if (m <= 64 && rows > sms) return {m <= 16 ? 16 : m <= 32 ? 32 : 64, 1, 2};
    static const struct { int bn, step, ends; } shapes[] = {
        {16, 220, 100}, {32, 220, 200}, {64, 210, 360}, {128, 290, 590}, {192, 350, 950}};
    static const struct { int bn, step, ends, least, start, part_step, part_ends; } pairs[] = {
        {192, 235, 455, 2745, 1180, 210, 1130}, {256, 275, 2600, 3100, 100, 225, 2250}};
    static const int join_start = 940, join_column[] = {0, 25, 27, 21};                          // CL = 1, 2, 4, 8
    GemmPlan best{256, 0};
    int64_t least = INT64_MAX;
    for (const auto &s : pairs) {
        if (m <= 64) break;
        const int64_t tiles = (n + 2 * BM - 1) / (2 * BM) * ((m + s.bn - 1) / s.bn), at_once = sms / 2;
        const bool cut = pair_parts(s.bn, tiles, at_once) > 1;
        const int64_t whole = cut ? tiles / at_once : (tiles + at_once - 1) / at_once;
        const int64_t round = steps * s.step + s.ends;
        const int64_t cost = s.start + whole * (round > s.least ? round : s.least) +
                             (cut && tiles % at_once ? steps * s.part_step + s.part_ends : 0);
        if (cost < least) {
            least = cost;
            best = {s.bn, 0};
        }
    }
    for (const auto &s : shapes) {
        if (s.bn < 64 && m > s.bn) continue;                      // narrow tiles start at a scale tile's first row
        if (s.bn > 16 && s.bn >= 2 * m) continue;
        const int64_t tiles = rows * ((m + s.bn - 1) / s.bn);
        for (int CL = 1, i = 0; CL <= 8 && CL <= steps; CL *= 2, ++i) {
            if (CL > 1 && s.bn > 128) break;                      // no room for partial sums
            const int64_t at_once = sms / CL - (CL == 8 ? sms / 32 : 0);   // GPCs hold few clusters of 8
            const int64_t rounds = (tiles + at_once - 1) / at_once;
            const int64_t cost = rounds * ((steps + CL - 1) / CL * s.step + s.ends +
                                           (CL > 1 ? join_start + (s.bn > 16 && m < s.bn ? m : s.bn) * join_column[i] : 0));
            if (cost < least) {
                least = cost;
                best = {s.bn, CL};
            }
        }
    }
    return best;
}

constexpr int OWN_STEPS = 16;       // steps of the activation that a CTA keeps
constexpr int OWN_TASKS = 32;       // token-steps that four warps quantize in less than a launch's time
constexpr int OWN_TASKS_LONG = 12;  // the same where two CTAs to an SM could take the quantizer's output

}  // namespace

GemmPlan gemm_mxfp4_plan(int sms, int64_t m, int64_t n, int64_t k) { return plan_tiles(sms, m, n, k); }

bool gemm_mxfp4_quantizes(int sms, int64_t m, int64_t n, int64_t k)
{
    const GemmPlan p = plan_tiles(sms, m, n, k);
    if (p.bn != 16) return false;                  // never pairs
    const int64_t steps = (k / BK + p.CL - 1) / p.CL;
    return steps <= OWN_STEPS && m * steps <= (p.per_sm == 2 ? OWN_TASKS_LONG : OWN_TASKS);
}

cudaError_t launch_gemm_mxfp4_own(const DeviceInfo &dev, const uint8_t *w, const uint8_t *wsc, const void *xf, int64_t ldx,
                                  int xtype, void *y, int type, int64_t m, int64_t n, int64_t k, cudaStream_t stream)
{
    return with_type(type, [&](auto t) {
        using T = decltype(t);
        return with_type(xtype, [&](auto u) {
            using X = decltype(u);
            return launch_tiles<Cfg<16, 8, OWN_STEPS>, T, X>(dev, w, wsc, nullptr, nullptr, static_cast<const X *>(xf), ldx,
                                                             static_cast<T *>(y), m, n, k, plan_tiles(dev.num_sms, m, n, k).CL,
                                                             false, stream);
        });
    });
}

cudaError_t launch_gemm_mxfp4(const DeviceInfo &dev, const uint8_t *w, const uint8_t *wsc, const uint8_t *x,
                              const uint8_t *xsc, void *y, int type, int64_t m, int64_t n, int64_t k, bool pdl,
                              cudaStream_t stream)
{
    return with_type(type, [&](auto t) {
        using T = decltype(t);
        T *out = static_cast<T *>(y);
        const GemmPlan p = plan_tiles(dev.num_sms, m, n, k);
        auto go = [&](auto cfg) {
            return launch_tiles<decltype(cfg), T, float>(dev, w, wsc, x, xsc, nullptr, 0, out, m, n, k, p.CL, pdl, stream);
        };
        auto pairs = [&](auto cfg) {
            return launch_pairs<decltype(cfg), T>(dev, w, wsc, x, xsc, out, m, n, k, pdl, stream);
        };
        if (p.CL == 0) return p.bn == 192 ? pairs(PairCfg<192>{}) : pairs(PairCfg<256>{});
        if (p.per_sm == 2)
            return p.bn == 16 ? go(Cfg<16, 5, 0, 2>{}) : p.bn == 32 ? go(Cfg<32, 5, 0, 2>{}) : go(Cfg<64, 4, 0, 2>{});
        if (p.bn == 16) return go(Cfg<16, 9>{});
        if (p.bn == 32) return go(Cfg<32, 8>{});
        if (p.bn == 64) return go(Cfg<64, 6>{});
        if (p.bn == 128) return go(Cfg<128, 4>{});
        return go(Cfg<192, 5>{});
    });
}

}  // namespace q8
