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
// Few output tiles (decode): the CTAs of a cluster split a tile's k among them.  Each sends its
// partial sums to the cluster's shared memories (rank c owns BN / CL of the tile's columns), and
// the owner adds them in rank order, so the result does not depend on timing.
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

template <int BN_, int STAGES_>
struct Cfg {
    static constexpr int BN = BN_;
    static constexpr int STAGES = STAGES_;
    static constexpr int NSB = BN > 128 ? 2 : 1;             // scale tiles that BN tokens touch
    static constexpr int B_BYTES = BN * ROW_BYTES;
    static constexpr bool SPLIT = BN <= 128;                 // room for the cluster's partial sums
    static constexpr int OFF_A = 0;
    static constexpr int OFF_B = OFF_A + STAGES * A_BYTES;
    static constexpr int OFF_SA = OFF_B + STAGES * B_BYTES;
    static constexpr int OFF_SB = OFF_SA + STAGES * SC_BYTES;
    static constexpr int OFF_RED = OFF_SB + STAGES * NSB * SC_BYTES;
    static constexpr int OFF_BAR = OFF_RED + (SPLIT ? BN * BM * 4 : 0);
    static constexpr int OFF_MISC = OFF_BAR + (2 * STAGES + 4 + 3) * 8;
    static constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;   // + slack for 1024-byte base alignment
    // Tensor memory: two accumulators, then two slots of scales (weights 8 columns, tokens 8 per
    // scale tile), so that a step's copies do not wait for the previous step's MMAs.
    static constexpr int SC_COLS = 8 + 8 * NSB;
    static constexpr int COL_SC = 2 * BN;
    static constexpr int NEED = COL_SC + 2 * SC_COLS;
    static constexpr int TMEM_COLS = NEED <= 64 ? 64 : NEED <= 128 ? 128 : NEED <= 256 ? 256 : 512;
    static_assert(NEED <= 512 && SMEM_BYTES <= SMEM_MAX, "capacity");
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
__device__ __forceinline__ void cluster_store(uint32_t addr, float v)
{
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void cluster_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// wait_or_abort whose success also orders what other CTAs of the cluster wrote before arriving.
__device__ __forceinline__ bool wait_cluster(uint64_t *bar, uint32_t parity, int *status, volatile int *abort_flag)
{
    const bool ok = wait_or_abort(bar, parity, status, abort_flag);
    asm volatile("fence.acq_rel.cluster;" ::: "memory");
    return ok;
}

struct Work {
    int m, n;
    int steps;        // k / BK
    int tiles;        // output tiles: token tile fastest
    int token_tiles;
    int first_wait;   // 1: the weights too may come from the kernel before this one
};

template <typename C, typename T>
__global__ void __launch_bounds__(THREADS, 1)
    gemm_mxfp4_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                      const uint8_t *__restrict__ wsc, const uint8_t *__restrict__ xsc, T *__restrict__ y, Work wk,
                      int CL, int *status)
{
    constexpr int BN = C::BN, STAGES = C::STAGES, NSB = C::NSB, B_BYTES = C::B_BYTES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
    uint64_t *empty = full + STAGES, *acc_full = empty + STAGES, *acc_empty = acc_full + 2;
    uint64_t *red_full = acc_empty + 2, *red_empty = red_full + 1, *drained = red_empty + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::OFF_MISC + 4);

    // Warp-uniform to the compiler too: the roles' loops then live in uniform registers.
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = CL > 1 ? cluster_rank() : 0;
    const int cluster = blockIdx.x / CL, clusters = gridDim.x / CL;
    const int ks0 = wk.steps * (int)rank / CL, ks1 = wk.steps * ((int)rank + 1) / CL;
    const int ktiles = wk.steps * (BK / MX_TILE_K);

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
        for (int s = 0; s < 2; ++s) { mbar_init(&acc_full[s], 1); mbar_init(&acc_empty[s], 4); }
        mbar_init(red_full, 4 * CL);
        mbar_init(red_empty, 4 * CL);
        mbar_init(drained, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 5) tc_alloc(tmem_slot, C::TMEM_COLS);
    if (warp == 4 && lane == 0) {
        prefetch_tensormap(&tm_w);
        prefetch_tensormap(&tm_x);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (CL > 1) cluster_sync_all();         // every rank's barriers exist before anyone arrives on them
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
            bytes = A_BYTES + B_BYTES + SC_BYTES * (1 + nsb);
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
                    load_x(st, ks);
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
        const uint64_t adesc0 = smem_desc_sw128(smem_u32(smem + C::OFF_A));
        const uint64_t bdesc0 = smem_desc_sw128(smem_u32(smem + C::OFF_B));
        const uint64_t sadesc0 = smem_desc_scales(smem_u32(smem + C::OFF_SA));
        const uint64_t sbdesc0 = smem_desc_scales(smem_u32(smem + C::OFF_SB));
        // Steps go in pairs where the second one's data is there: the tensor pipe runs copies and
        // MMAs in order and pays for each change between them.
        auto copy_scales = [&](int slot, int st) {
            const uint32_t sa = tmem + C::COL_SC + slot * C::SC_COLS, sb = sa + 8;
#pragma unroll
            for (int g = 0; g < 2; ++g) {        // the step's two groups of 128 values
                tc_copy_scales(sa + 4 * g, sadesc0 + (uint64_t)((st * SC_BYTES + g * MX_TILE_BYTES) >> 4));
#pragma unroll
                for (int b = 0; b < NSB; ++b)
                    tc_copy_scales(sb + 4 * (NSB * g + b),
                                   sbdesc0 + (uint64_t)(((st * NSB + b) * SC_BYTES + g * MX_TILE_BYTES) >> 4));
            }
        };
        auto multiply = [&](int slot, int st, uint32_t d_tmem, uint32_t sb_shift, bool first) {
            const uint32_t sa = tmem + C::COL_SC + slot * C::SC_COLS, sb = sa + 8 + sb_shift;
            const uint64_t ad = adesc0 + (uint64_t)(st * (A_BYTES >> 4));
            const uint64_t bd = bdesc0 + (uint64_t)(st * (B_BYTES >> 4));
#pragma unroll
            for (int j = 0; j < 4; ++j) {        // 64 values: bytes 2 (j % 2) and next of each scale word
                const uint32_t id = C::IDESC | ((uint32_t)(2 * (j & 1)) << 4) | ((uint32_t)(2 * (j & 1)) << 29);
                tc_mma_mxf4(d_tmem, ad + 2 * j, bd + 2 * j, id, sa + 4 * (j >> 1), sb + 4 * NSB * (j >> 1), !first || j > 0);
            }
            tc_commit(&empty[st]);
        };
        int st = 0, i = 0;
        uint32_t phase = 0;
        bool ok = true;
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
                    copy_scales(0, st);
                    if (two) copy_scales(1, st1);
                    multiply(0, st, tmem + acc * BN, sb_shift, ks == ks0);
                    if (two) multiply(1, st1, tmem + acc * BN, sb_shift, false);
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
        int i = 0;
        for (int tile = cluster; tile < wk.tiles; tile += clusters, ++i) {
            const int acc = i & 1;
            const int64_t r = (int64_t)(tile / wk.token_tiles) * BM + row;
            const int tok0 = tile % wk.token_tiles * BN;
            const int cols = min(BN, wk.m - tok0);
            if (!__all_sync(0xffffffffu, wait_or_abort(&acc_full[acc], (i >> 1) & 1, status, abort_flag))) break;
            tc_fence_after();
            T *dst = y + (int64_t)tok0 * wk.n + r;
            if (CL == 1) {
#pragma unroll 1
                for (int c0 = 0; c0 < cols; c0 += 16) {
                    uint32_t v[16];
                    tc_ld_x16(tmem + lane_base + acc * BN + c0, v);
                    if (r < wk.n)
#pragma unroll
                        for (int c = 0; c < 16; ++c)
                            if (c0 + c < cols) dst[(int64_t)(c0 + c) * wk.n] = from_f32<T>(__uint_as_float(v[c]));
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&acc_empty[acc]);
            } else if constexpr (C::SPLIT) {
                const int per = BN / CL;                                // columns that a rank owns
                if (!__all_sync(0xffffffffu, wait_cluster(red_empty, (i & 1) ^ 1, status, abort_flag))) break;
#pragma unroll 1
                for (int c0 = 0; c0 < cols; c0 += 16) {
                    uint32_t v[16];
                    tc_ld_x16(tmem + lane_base + acc * BN + c0, v);
#pragma unroll
                    for (int c = 0; c < 16; ++c)
                        if (c0 + c < cols) {
                            const int owner = (c0 + c) / per, at = (c0 + c) % per;
                            cluster_store(cluster_addr(smem_u32(red + ((int)rank * per + at) * BM + row), owner),
                                          __uint_as_float(v[c]));
                        }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&acc_empty[acc]);
                    for (int c = 0; c < CL; ++c) cluster_arrive(cluster_addr(smem_u32(red_full), c));
                }
                if (!__all_sync(0xffffffffu, wait_cluster(red_full, i & 1, status, abort_flag))) break;
                const int own0 = (int)rank * per;
                for (int c = 0; c < per && own0 + c < cols; ++c) {
                    float s = red[c * BM + row];
                    for (int src = 1; src < CL; ++src) s += red[(src * per + c) * BM + row];
                    if (r < wk.n) dst[(int64_t)(own0 + c) * wk.n] = from_f32<T>(s);
                }
                __syncwarp();
                if (lane == 0)
                    for (int c = 0; c < CL; ++c) cluster_arrive(cluster_addr(smem_u32(red_empty), c));
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (CL > 1) cluster_sync_all();         // nobody leaves while others may still write to it
    if (warp == 5) {
        tc_fence_after();
        tc_dealloc(tmem, C::TMEM_COLS);
    }
}

// Clusters of CL CTAs that are resident at once (looked up once per device, kernel and CL).
template <typename C, typename T>
cudaError_t resident_clusters(const DeviceInfo &dev, int CL, int *count)
{
    static std::atomic<int> known[kAttrDevices][4];
    const int slot = CL == 1 ? 0 : CL == 2 ? 1 : CL == 4 ? 2 : 3;
    const bool cache = dev.device >= 0 && dev.device < kAttrDevices;
    if (CL == 1) {
        *count = dev.num_sms;
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
    cudaError_t e = cudaOccupancyMaxActiveClusters(&got, gemm_mxfp4_kernel<C, T>, &cfg);
    if (e != cudaSuccess) return e;
    *count = got < dev.num_sms / CL ? got : dev.num_sms / CL;
    if (*count < 1) return cudaErrorInvalidConfiguration;
    if (cache) known[dev.device][slot].store(*count, std::memory_order_relaxed);
    return cudaSuccess;
}

template <typename C, typename T>
cudaError_t launch_tiles(const DeviceInfo &dev, const uint8_t *w, const uint8_t *wsc, const uint8_t *x,
                         const uint8_t *xsc, T *y, int64_t m, int64_t n, int64_t k, int CL, bool pdl, cudaStream_t stream)
{
    cudaError_t e = set_kernel_smem<gemm_mxfp4_kernel<C, T>>(dev.device, C::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    int resident = 0;
    if ((e = resident_clusters<C, T>(dev, CL, &resident)) != cudaSuccess) return e;
    CUtensorMap tm_w, tm_x;
    if (!encode_2d(&tm_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, w, (uint64_t)k / 2, (uint64_t)n, (uint64_t)k / 2, ROW_BYTES, BM,
                   CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_2d(&tm_x, CU_TENSOR_MAP_DATA_TYPE_UINT8, x, (uint64_t)k / 2, (uint64_t)m, (uint64_t)k / 2, ROW_BYTES,
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
    return cudaLaunchKernelEx(&cfg, gemm_mxfp4_kernel<C, T>, tm_w, tm_x, wsc, xsc, y, wk, CL, dev.status);
}

}  // namespace

cudaError_t launch_gemm_mxfp4(const DeviceInfo &dev, const uint8_t *w, const uint8_t *wsc, const uint8_t *x,
                              const uint8_t *xsc, void *y, int type, int64_t m, int64_t n, int64_t k, bool pdl,
                              cudaStream_t stream)
{
    return with_type(type, [&](auto t) {
        using T = decltype(t);
        T *out = static_cast<T *>(y);
        // As many CTAs to a tile as leave no more than one wave, each with a step at least.
        const int64_t rows = (n + BM - 1) / BM;
        auto split = [&](int bn) {
            const int64_t tiles = rows * ((m + bn - 1) / bn);
            int CL = 1;
            while (CL < 8 && tiles * CL * 2 <= dev.num_sms && CL * 2 <= k / BK) CL *= 2;
            return CL;
        };
        if (m <= 16) return launch_tiles<Cfg<16, 9>, T>(dev, w, wsc, x, xsc, out, m, n, k, split(16), pdl, stream);
        if (m <= 32) return launch_tiles<Cfg<32, 8>, T>(dev, w, wsc, x, xsc, out, m, n, k, split(32), pdl, stream);
        if (m <= 64) return launch_tiles<Cfg<64, 6>, T>(dev, w, wsc, x, xsc, out, m, n, k, split(64), pdl, stream);
        if (m <= 128) return launch_tiles<Cfg<128, 4>, T>(dev, w, wsc, x, xsc, out, m, n, k, split(128), pdl, stream);
        return launch_tiles<Cfg<192, 5>, T>(dev, w, wsc, x, xsc, out, m, n, k, 1, pdl, stream);
    });
}

}  // namespace q8
