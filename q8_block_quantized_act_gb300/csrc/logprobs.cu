// logprobs.cu -- for each row of logits: the log probability of a given token, the entropy of
// the softmax, and the most likely tokens with their log probabilities.
//   mx = max x,  S = sum e^(x - mx),  T = sum (x - mx) e^(x - mx)
//   log p(i) = x_i - mx - log S,      H = log S - T / S
// A row whose logits are all -inf has no distribution: log probabilities -inf, entropy 0, no
// alternatives (id -1).  A row with a NaN or +inf: NaN everywhere, ids -1.
//
// Bound by memory for many rows: 509 rows of 128896 bf16 take 24.3 us without alternatives, 28.2
// with 8 (19.4 by bytes; 3.3 CTAs to an SM).  The loads' latency is covered by 2 x 16 KB on their way
// to each CTA's shared memory (a step ahead in registers alone: 26.6 us).  One row: 6.0 us, latency
// (the pass 3.3, ranking and the cluster's join 2.7).
//
// One pass over the row.  Every thread keeps its own running maximum, S and T (f32) of the
// 16-byte vectors it owns, rescaled when its maximum rises, and stores the maximum of each slot of
// its steps.  The threads' maxima give a bound that at least `top` logits reach; afterwards only the
// few slots whose maximum reaches it are read again (from L2), and the keys (logit, index) found
// there are ranked by counting.  Where more slots than the list has places reach it (rows of equal
// logits, or all but a few at the type's lowest value), the warps go over the row once more with
// sorted lists in registers, skipping what cannot enter them.
// Few rows: a cluster of CTAs shares a row and joins its parts through distributed shared memory.
#include "launch.h"
#include "types.cuh"

namespace q8 {
namespace {

constexpr unsigned ALL = 0xffffffffu;
constexpr int U = 4;              // vectors of a step per thread
constexpr int RING = 2;           // steps on their way to shared memory
constexpr int MAX_CL = 8;
constexpr int CAP = 256;          // keys that the CTA's list holds
constexpr int MAX_J = 8;
constexpr int SLOTS = 16;         // maxima kept of each thread's steps
constexpr float LOG2E = 1.44269504f;
constexpr float LOWEST = -3.4028235e38f;

// Larger logits and, among equal ones, lower indexes have larger keys; 0 is below every key.
__device__ __forceinline__ uint32_t order_of(float x)
{
    const uint32_t b = __float_as_uint(x == 0.0f ? 0.0f : x);      // -0 and +0 are equal
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t key_of(float x, uint32_t i) { return ((uint64_t)order_of(x) << 32) | (uint32_t)~i; }
__device__ __forceinline__ float value_of(uint64_t key)
{
    const uint32_t o = (uint32_t)(key >> 32);
    return __uint_as_float((o & 0x80000000u) ? o & 0x7fffffffu : ~o);
}

// 2^x, results below the normal numbers as 0 (they count nothing against a sum of 1 at least;
// keeping them takes three more instructions for each element).
__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// ---- lists of 32 keys, one a lane, largest first ----
__device__ __forceinline__ void exchange(uint64_t &k, int o, bool larger)
{
    const uint64_t other = __shfl_xor_sync(ALL, k, o);
    k = (k > other) == larger ? k : other;
}
// The 32 largest of two lists (a bitonic sequence, then its five half-cleaners).
__device__ __forceinline__ void merge32(uint64_t &k, uint64_t other, int lane)
{
    const uint64_t rev = __shfl_sync(ALL, other, 31 - lane);
    k = k > rev ? k : rev;
#pragma unroll
    for (int o = 16; o; o >>= 1) exchange(k, o, (lane & o) == 0);
}
__device__ __forceinline__ void insert32(uint64_t &k, uint64_t c, int lane)
{
    const int pos = __popc(__ballot_sync(ALL, k > c));
    const uint64_t up = __shfl_up_sync(ALL, k, 1);
    k = lane == pos ? c : lane > pos ? up : k;
}

// Softmax statistics relative to m.
struct Stats {
    float m, s, t;
};
// The same sums relative to m >= a.m.
__device__ __forceinline__ void rescale(Stats &a, float m)
{
    const float d = fmaxf(a.m - m, LOWEST), f = ex2(d * LOG2E);
    a.t = f > 0.0f ? f * fmaf(a.s, d, a.t) : 0.0f;
    a.s *= f;
    a.m = m;
}

// The sums of n <= 32 parts, one a lane, in a fixed order.
__device__ __forceinline__ Stats join(Stats a)
{
    float mx = a.m;
#pragma unroll
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(ALL, mx, o));
    rescale(a, mx);
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        a.s += __shfl_xor_sync(ALL, a.s, o);
        a.t += __shfl_xor_sync(ALL, a.t, o);
    }
    return a;
}

// A vector of masked logits.
template <typename T>
__device__ __forceinline__ uint4 none()
{
    const uint32_t w = sizeof(T) == 4 ? 0xff800000u : std::is_same<T, __half>::value ? 0xfc00fc00u : 0xff80ff80u;
    return make_uint4(w, w, w, w);
}

// The largest element of N vectors (NaN ignored).
template <typename T, int N>
__device__ __forceinline__ float largest(const uint4 (&r)[N])
{
    float f[VEC<T>];
    if constexpr (sizeof(T) == 4) {
        float mx = __int_as_float(0xff800000);
#pragma unroll
        for (int u = 0; u < N; ++u) {
            unpack<T>(r[u], f);
            mx = fmaxf(mx, fmaxf(fmaxf(f[0], f[1]), fmaxf(f[2], f[3])));
        }
        return mx;
    } else {
        using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
        T2 mx = *reinterpret_cast<const T2 *>(&r[0].x);
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const uint32_t w[4] = {r[u].x, r[u].y, r[u].z, r[u].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) mx = __hmax2(mx, *reinterpret_cast<const T2 *>(&w[i]));
        }
        return fmaxf(to_f32(mx.x), to_f32(mx.y));
    }
}

template <int W>
struct Shared {
    union {
        uint4 ring[RING][U][W * 32];       // each thread its own vectors
        int chosen[SLOTS * W * 32];        // after the pass: (thread, slot) pairs whose maximum reaches the bound
    };
    uint64_t list[W][32];
    uint64_t found[CAP];               // keys that reach the bound, in no order
    Stats stats[W];
    float slot[SLOTS][W * 32];         // each thread's maxima
    uint32_t best[W * MAX_J];          // each warp's J largest thread maxima
    uint32_t bound;
    int n_chosen, n_found;
    uint64_t part_list[MAX_CL][32];    // rank 0: every rank's list and sums
    Stats part_stats[MAX_CL];
};

__device__ __forceinline__ void copy16_async(void *dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ uint32_t remote(const void *p, uint32_t rank)
{
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}

// n (a power of two) lists to one, pairwise: warp w takes over list w + half.
__device__ __forceinline__ void join_lists(uint64_t (*lists)[32], int n, uint64_t &list, int warp, int lane)
{
    for (int half = n / 2; half; half >>= 1) {
        if (warp < half) {
            merge32(list, lists[warp + half][lane], lane);
            lists[warp][lane] = list;
        }
        __syncthreads();
    }
}

template <typename T, int THREADS>
__global__ void __launch_bounds__(THREADS, 4) logprobs_kernel(LogprobArgs a, int64_t m, int v, int CL)
{
    constexpr int V = VEC<T>, W = THREADS / 32;
    extern __shared__ __align__(16) uint8_t smem[];
    Shared<W> &sh = *reinterpret_cast<Shared<W> *>(smem);
    const float ninf = __int_as_float(0xff800000), nan = __int_as_float(0x7fffffff);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t rank = 0;
    if (CL > 1) {
        asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
        asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");   // this CTA runs
    }
    if (threadIdx.x == 0) sh.n_chosen = sh.n_found = 0;
    griddep_enter();
    // CL > 1: one row per cluster (the grid holds them all)
    for (int64_t row = blockIdx.x / CL; row < m; row += gridDim.x / CL) {
        const T *x = static_cast<const T *>(a.logits) + row * a.ld;
        // The row's whole 16-byte vectors, of which this CTA has [L0, L1); up to V - 1 elements at
        // either end are left over (edges), one for each of rank 0's first threads.
        const int lead = (int)((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));
        const int head = lead ? min(V - lead, v) : 0, whole = (v - head) / V, tail = v - head - whole * V;
        const uint4 *vec = reinterpret_cast<const uint4 *>(x + head);
        const int L0 = (int)((int64_t)whole * rank / CL), L1 = (int)((int64_t)whole * (rank + 1) / CL);

        // ---- the pass: two steps' vectors are on their way while a step is summed ----
        Stats st{LOWEST, 0.0f, 0.0f};
        float2 sum = make_float2(0.0f, 0.0f), tsum = make_float2(0.0f, 0.0f);   // two partial sums each
        constexpr int STEP = U * THREADS;                            // vectors of a step
        const int steps = (L1 - L0 + STEP - 1) / STEP, per_slot = (steps + SLOTS - 1) / SLOTS;
        auto fetch = [&](int step) {
            const int L = L0 + step * STEP + (int)threadIdx.x;
            uint4 (*to)[THREADS] = sh.ring[step % RING];
            if (L0 + (step + 1) * STEP <= L1) {
#pragma unroll
                for (int u = 0; u < U; ++u) copy16_async(&to[u][threadIdx.x], vec + L + u * THREADS);
            } else if (step < steps) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (L + u * THREADS < L1) copy16_async(&to[u][threadIdx.x], vec + L + u * THREADS);
                    else to[u][threadIdx.x] = none<T>();
                }
            }
            copies_commit();
        };
#pragma unroll
        for (int i = 0; i < RING; ++i) fetch(i);
        float edge = ninf;                                           // its element is edge_at
        const int edge_at = (int)threadIdx.x < head ? (int)threadIdx.x : v - tail + (int)threadIdx.x - head;
        if (rank == 0 && (int)threadIdx.x < head + tail) {
            edge = to_f32(x[edge_at]);
            st = edge > ninf ? Stats{edge, 1.0f, 0.0f} : st;
            if (!(edge < __int_as_float(0x7f800000))) st.s = nan;
            sum.x = st.s;
        }
        int left = per_slot, slots = 0;
        float slot_max = ninf;
        for (int step = 0; step < steps; ++step) {
            uint4 cur[U];
            copies_wait<RING - 1>();
#pragma unroll
            for (int u = 0; u < U; ++u) cur[u] = sh.ring[step % RING][u][threadIdx.x];
            const float mx = largest<T, U>(cur);                         // every vector has been read
            fetch(step + RING);
            slot_max = fmaxf(slot_max, mx);
            if (--left == 0 || step + 1 == steps) {
                sh.slot[slots++][threadIdx.x] = slot_max;
                slot_max = ninf;
                left = per_slot;
            }
            if (mx > st.m) {
                Stats lo{st.m, sum.x, tsum.x}, hi{st.m, sum.y, tsum.y};
                rescale(lo, mx);
                rescale(hi, mx);
                sum = make_float2(lo.s, hi.s);
                tsum = make_float2(lo.t, hi.t);
                st.m = mx;
            }
            const float2 neg = make_float2(-st.m, -st.m);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float f[V];
                unpack<T>(cur[u], f);
#pragma unroll
                for (int j = 0; j < V; j += 2) {
                    const float2 z = __fadd2_rn(make_float2(f[j], f[j + 1]), neg);
                    const float2 p = __fmul2_rn(z, make_float2(LOG2E, LOG2E));
                    const float2 e = make_float2(ex2(p.x), ex2(p.y));
                    sum = __fadd2_rn(sum, e);                     // a NaN or +inf makes it NaN
                    // masked: 0 times a finite number
                    tsum = __ffma2_rn(make_float2(fmaxf(z.x, LOWEST), fmaxf(z.y, LOWEST)), e, tsum);
                }
            }
        }
        st.s = sum.x + sum.y;
        st.t = tsum.x + tsum.y;
        float asked = 0.0f;
        int32_t token = -1;
        if (a.tokens && threadIdx.x == 0 && rank == 0) {
            token = a.tokens[row];
            if (token >= 0 && token < v) asked = to_f32(x[token]);
        }

        // ---- a bound that `top` logits reach: the top-th of the warps' J largest thread maxima ----
        const uint32_t own = st.s > 0.0f ? order_of(st.m) : 0;      // 0: nothing but masked logits
        const int J = min((a.top + W - 1) / W + 2, MAX_J);
        if (a.top > 0) {
            uint32_t k = own;
#pragma unroll 1
            for (int i = 0; i < J; ++i) {
                const uint32_t best = __reduce_max_sync(ALL, k);
                if (lane == __ffs(__ballot_sync(ALL, k == best)) - 1) {
                    sh.best[warp * J + i] = best;
                    k = 0;
                }
            }
        }
        st = join(st);
        if (lane == 0) sh.stats[warp] = st;
        __syncthreads();

        // ---- the alternatives ----
        uint64_t list = 0;
        if (a.top > 0) {
            // the first warp ranks the W J <= 64 values, two a lane, equal ones by their place
            if (warp == 0) {
                uint32_t mine[2] = {0, 0};
                int place[2] = {0, 0};
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (lane + 32 * h < W * J) mine[h] = sh.best[lane + 32 * h];
#pragma unroll 8
                for (int i = 0; i < W * J; ++i) {
                    const uint32_t other = sh.best[i];
#pragma unroll
                    for (int h = 0; h < 2; ++h) place[h] += other > mine[h] || (other == mine[h] && i < lane + 32 * h);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (place[h] == a.top - 1 && lane + 32 * h < W * J) sh.bound = mine[h];
            }
            __syncthreads();
            uint32_t thr = sh.bound;
            thr = max(thr, 1u);
            const float least = thr > 1u ? value_of((uint64_t)thr << 32) : LOWEST;
            sh.list[warp][lane] = 0;
            uint32_t reach = 0;
            if (own >= thr) {
#pragma unroll
                for (int i = 0; i < SLOTS; ++i)
                    if (i < slots) reach |= (sh.slot[i][threadIdx.x] >= least ? 1u : 0u) << i;
                if (edge >= least) {
                    const int n = atomicAdd(&sh.n_found, 1);
                    if (n < CAP) sh.found[n] = key_of(edge, (uint32_t)edge_at);
                }
            }
            if (__any_sync(ALL, reach != 0)) {
                int upto = __popc(reach);
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int below = __shfl_up_sync(ALL, upto, o);
                    if (lane >= o) upto += below;
                }
                int at = 0;
                if (lane == 31) at = atomicAdd(&sh.n_chosen, upto);
                at = __shfl_sync(ALL, at, 31) + upto - __popc(reach);
                for (; reach; reach &= reach - 1) sh.chosen[at++] = (int)threadIdx.x * SLOTS + __ffs(reach) - 1;
            }
            __syncthreads();
            // Each warp reads the U V elements of a chosen thread's step, one a lane (f32: two
            // steps at once), several in flight.
            constexpr int LANES = U * V, AT_ONCE = 32 / LANES, DEPTH = 8 / AT_ONCE;
            const int pairs = sh.n_chosen;                            // each holds a key: more than CAP is too many
            const int scan = pairs <= CAP ? pairs * per_slot : 0;
#pragma unroll 1
            for (int i0 = warp * AT_ONCE; i0 < scan; i0 += W * AT_ONCE * DEPTH) {
                // per_slot is 1 up to SLOTS steps; longer rows go over a slot's steps one by one
                float f[DEPTH];
                int at[DEPTH];
#pragma unroll
                for (int d = 0; d < DEPTH; ++d) {
                    const int i = i0 + d * W * AT_ONCE + lane / LANES;
                    f[d] = ninf;
                    at[d] = 0;
                    if (i < scan) {
                        const int pair = sh.chosen[per_slot == 1 ? i : i / per_slot];
                        const int step = per_slot == 1 ? pair % SLOTS : pair % SLOTS * per_slot + i % per_slot;
                        const int L = L0 + step * STEP + pair / SLOTS + lane % LANES / V * THREADS;
                        at[d] = head + L * V + lane % V;
                        if (L < L1) f[d] = to_f32(x[at[d]]);
                    }
                }
#pragma unroll
                for (int d = 0; d < DEPTH; ++d)
                    if (f[d] >= least) {
                        const int n = atomicAdd(&sh.n_found, 1);
                        if (n < CAP) sh.found[n] = key_of(f[d], (uint32_t)at[d]);
                    }
            }
            __syncthreads();
            const int n = pairs <= CAP ? sh.n_found : CAP + 1;
            if (n <= CAP) {
                // A key's place is the number of larger ones; the keys differ, so places do.
                if ((int)threadIdx.x < n) {
                    const uint64_t k = sh.found[threadIdx.x];
                    int place = 0;
#pragma unroll 1
                    for (int i = 0; i < n; i += 8)
#pragma unroll
                        for (int j = 0; j < 8; ++j) place += i + j < n && sh.found[i + j] > k;
                    if (place < 32) sh.list[0][place] = k;
                }
                __syncthreads();
                list = sh.list[0][lane];
            } else {
                auto offer = [&](float f, int at) {
                    const uint64_t k = key_of(f, (uint32_t)at);
                    const uint64_t worst = __shfl_sync(ALL, list, a.top - 1);
                    unsigned some = __ballot_sync(ALL, f >= least && k > worst);
                    for (; some; some &= some - 1) insert32(list, __shfl_sync(ALL, k, __ffs(some) - 1), lane);
                };
                // A warp goes through its elements by rising index (the tail last), 32 vectors at a
                // time: once its list is full, a group without a larger logit than the list's last
                // has nothing for it, equal ones included.
                if (warp == 0) offer((int)threadIdx.x < head ? edge : ninf, edge_at);
#pragma unroll 1
                for (int base = L0 + warp * 32; base < L1; base += U * THREADS) {
                    uint4 r[U];
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const int L = base + u * THREADS + lane;
                        r[u] = L < L1 ? __ldg(vec + L) : none<T>();
                    }
#pragma unroll 1
                    for (int u = 0; u < U; ++u) {
                        const uint4 one[1] = {r[0]};
#pragma unroll
                        for (int i = 0; i + 1 < U; ++i) r[i] = r[i + 1];
                        const float mx = largest<T, 1>(one);
                        const uint64_t last = __shfl_sync(ALL, list, a.top - 1);
                        if (!__any_sync(ALL, mx >= least && (last == 0 || mx > value_of(last)))) continue;
                        float f[V];
                        unpack<T>(one[0], f);
                        const int at = head + (base + u * THREADS + lane) * V;
#pragma unroll
                        for (int j = 0; j < V; ++j) offer(f[j], at + j);
                    }
                }
                if (warp == 0) offer((int)threadIdx.x >= head ? edge : ninf, edge_at);
                sh.list[warp][lane] = list;
                __syncthreads();
                join_lists(sh.list, W, list, warp, lane);
            }
        }

        // ---- join the warps' sums, then the cluster's parts ----
        Stats all{LOWEST, 0.0f, 0.0f};
        if (warp == 0) {
            if (lane < W) all = sh.stats[lane];
            all = join(all);
        }
        if (CL > 1) {
            asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");       // rank 0 runs
            if (warp == 0) {
                if (a.top > 0)
                    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(remote(&sh.part_list[rank][lane], 0)), "l"(list)
                                 : "memory");
                if (lane == 0) {
                    const uint32_t to = remote(&sh.part_stats[rank], 0);
                    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(all.m) : "memory");
                    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + 4), "f"(all.s) : "memory");
                    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + 8), "f"(all.t) : "memory");
                }
            }
            asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
            if (rank == 0) {
                if (a.top > 0) {
                    if (warp < CL) list = sh.part_list[warp][lane];
                    join_lists(sh.part_list, CL, list, warp, lane);
                }
                if (warp == 0) {
                    all = Stats{LOWEST, 0.0f, 0.0f};
                    if (lane < CL) all = sh.part_stats[lane];
                    all = join(all);
                }
            }
        }
        if (warp == 0) {
            if (rank == 0) {
                const bool bad = !(all.s >= 0.0f), empty = all.s == 0.0f;
                const float lse = logf(all.s), mxr = all.m;
                if (lane == 0) {
                    if (a.entropy) a.entropy[row] = bad ? nan : empty ? 0.0f : lse - all.t / all.s;
                    if (a.logprob)
                        a.logprob[row] = token < 0 ? 0.0f : token >= v || bad ? nan : empty ? ninf : (asked - mxr) - lse;
                }
                if (lane < a.top) {
                    a.top_ids[row * a.top + lane] = bad || list == 0 ? -1 : (int32_t)~(uint32_t)list;
                    a.top_logprobs[row * a.top + lane] = bad ? nan : list == 0 ? ninf : (value_of(list) - mxr) - lse;
                }
            }
        }
        if (threadIdx.x == 0) sh.n_chosen = sh.n_found = 0;       // read by everyone before the last barrier
        __syncthreads();
    }
}

template <typename T, int THREADS>
cudaError_t launch_rows(const DeviceInfo &dev, const LogprobArgs &a, int64_t m, int64_t v, int CL, cudaStream_t stream)
{
    const int64_t rows = CL > 1 || m < (1 << 24) ? m : (1 << 24);
    cudaLaunchConfig_t cfg = {};
    constexpr size_t smem = sizeof(Shared<THREADS / 32>);
    const cudaError_t e = set_kernel_smem<logprobs_kernel<T, THREADS>>(dev.device, smem);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3((unsigned)(rows * CL));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)CL;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CL > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, logprobs_kernel<T, THREADS>, a, m, (int)v, CL);
}

}  // namespace

cudaError_t launch_logprobs(const DeviceInfo &dev, const LogprobArgs &a, int64_t m, int64_t v, int type,
                            cudaStream_t stream)
{
    return with_type(type, [&](auto t) {
        using T = decltype(t);
        constexpr int THREADS = 256;
        // Share a row of three steps or more among CTAs while each keeps half a step as long as they
        // have an SM each, two steps up to 7 CTAs on 4 SMs, four up to 2 on one (0.4 % above the best of
        // 1, 2, 4 and 8 on average over 340 sizes; 76 x 128896 bf16 with 8 alternatives: 11.6 us not
        // shared, 10.1 by two, 13.1 by four; 32 x 8192 f32: 4.4 not shared, 5.7 by eight).
        const int64_t step = U * THREADS, vecs = v / VEC<T>;
        int CL = 1;
        while (CL < MAX_CL && vecs >= 3 * step) {
            const int64_t ctas = m * CL * 2, sms = dev.num_sms;
            const int64_t least = ctas <= sms ? step / 2 : ctas * 4 <= sms * 7 ? 2 * step : 4 * step;
            if (ctas > 2 * sms || vecs / (CL * 2) < least) break;
            CL *= 2;
        }
        return launch_rows<T, THREADS>(dev, a, m, v, CL, stream);
    });
}

}  // namespace q8
