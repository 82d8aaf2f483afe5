// logprobs.cu -- for each row of logits: the log probability of a given token, the entropy of
// the softmax, and the most likely tokens with their log probabilities.
//   mx = max x,  S = sum e^(x - mx),  T = sum (x - mx) e^(x - mx)
//   log p(i) = x_i - mx - log S,      H = log S - T / S
// A row whose logits are all -inf has no distribution: log probabilities -inf, entropy 0, no
// alternatives (id -1).  A row with a NaN or +inf: NaN everywhere, ids -1.
//
// One pass over the row.  Every thread keeps its own running maximum, S and T (f32) of the
// 16-byte vectors it owns, rescaled when its maximum rises.  The alternatives cost nothing in
// that pass: of each thread's maximum and the place where it rose, a bound follows that at least
// `top` of the row's (logit, index) keys reach, and afterwards only the few threads whose maximum
// reaches it have their vectors read again (from L2).
// Few rows: a cluster of CTAs shares a row and joins its parts through distributed shared memory.
#include "launch.h"
#include "types.cuh"

namespace q8 {
namespace {

constexpr unsigned ALL = 0xffffffffu;
constexpr int U = 4;              // vectors in flight per thread
constexpr int MAX_CL = 8;
constexpr float LOG2E = 1.44269504f, LN2 = 0.693147181f;
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

__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// ---- lists of 32 keys, one a lane, largest first ----
__device__ __forceinline__ void exchange(uint64_t &k, int o, bool larger)
{
    const uint64_t other = __shfl_xor_sync(ALL, k, o);
    k = (k > other) == larger ? k : other;
}
__device__ __forceinline__ void sort32(uint64_t &k, int lane)
{
#pragma unroll
    for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
        for (int o = size / 2; o; o >>= 1) exchange(k, o, ((lane & o) == 0) == ((lane & size) == 0));
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

// The row on the grid of 16-byte vectors: vector L holds elements L V - lead .. + V - 1, of which
// the first and the last vector may have only some.
template <typename T>
struct Row {
    const T *x;          // the row's first element
    int lead, v;
    __device__ __forceinline__ int vectors() const { return (lead + v + VEC<T> - 1) / VEC<T>; }
    __device__ __forceinline__ void load(int L, float (&f)[VEC<T>]) const
    {
        const int e0 = L * VEC<T> - lead;
        if (e0 >= 0 && e0 + VEC<T> <= v) {
            unpack<T>(__ldg(reinterpret_cast<const uint4 *>(x + e0)), f);
        } else {
#pragma unroll
            for (int j = 0; j < VEC<T>; ++j)
                f[j] = e0 + j >= 0 && e0 + j < v ? to_f32(x[e0 + j]) : __int_as_float(0xff800000);
        }
    }
};

template <int W>
struct Shared {
    uint64_t list[W][32];
    Stats stats[W];
    uint64_t bound[W];
    uint64_t part_list[MAX_CL][32];    // rank 0: every rank's list and sums
    Stats part_stats[MAX_CL];
};

__device__ __forceinline__ uint32_t remote(const void *p, uint32_t rank)
{
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}

template <typename T, int THREADS>
__global__ void __launch_bounds__(THREADS) logprobs_kernel(LogprobArgs a, int64_t m, int v, int CL)
{
    constexpr int V = VEC<T>, W = THREADS / 32;
    __shared__ Shared<W> sh;
    const float ninf = __int_as_float(0xff800000), nan = __int_as_float(0x7fffffff);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t rank = 0;
    if (CL > 1) {
        asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
        asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");   // this CTA runs
    }
    griddep_enter();
    // CL > 1: one row per cluster (the grid holds them all)
    for (int64_t row = blockIdx.x / CL; row < m; row += gridDim.x / CL) {
        Row<T> x;
        x.x = static_cast<const T *>(a.logits) + row * a.ld;
        x.lead = (int)((reinterpret_cast<uintptr_t>(x.x) & 15u) / sizeof(T));
        x.v = v;
        const int64_t nv = x.vectors();
        const int L0 = (int)(nv * rank / CL), L1 = (int)(nv * (rank + 1) / CL);
        int32_t token = -1;
        float asked = 0.0f;
        if (a.tokens && threadIdx.x == 0 && rank == 0) {
            token = a.tokens[row];
            if (token >= 0 && token < v) asked = to_f32(x.x[token]);
        }

        // ---- the pass ----
        Stats st{LOWEST, 0.0f, 0.0f};
        int rose = 0;                      // the step in which this thread's maximum rose last
        int step = 0;
        for (int L = L0 + (int)threadIdx.x; L < L1; L += U * THREADS, ++step) {
            float f[U][V];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (L + u * THREADS < L1) {
                    x.load(L + u * THREADS, f[u]);
                } else {
#pragma unroll
                    for (int j = 0; j < V; ++j) f[u][j] = ninf;
                }
            }
            float mx = f[0][0];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int j = 0; j < V; ++j) mx = fmaxf(mx, f[u][j]);
            if (mx > st.m || (step == 0 && mx > ninf)) {
                rescale(st, fmaxf(mx, st.m));
                rose = step;
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float z = f[u][j] - st.m, e = ex2(z * LOG2E);
                    st.s += e;                                    // a NaN or +inf makes it NaN
                    st.t = fmaf(fmaxf(z, LOWEST), e, st.t);       // masked: 0 times a finite number
                }
        }

        // ---- a bound that `top` keys reach: in each warp, top / W of its threads' maxima ----
        const bool live = st.s > 0.0f;
        uint64_t thr = 0;
        if (a.top > 0) {
            // no smaller than the index of the element that holds the maximum
            const int64_t last = ((int64_t)L0 + threadIdx.x + ((int64_t)rose * U + U) * THREADS) * V;
            uint64_t k = live ? key_of(st.m, (uint32_t)(last < v ? last : v)) : 0;
            sort32(k, lane);
            const int per = (a.top + W - 1) / W;
            if (lane == per - 1) sh.bound[warp] = k;
        }
        // ---- the CTA's sums ----
        const float own_m = st.m;
        float mx = st.m;
#pragma unroll
        for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(ALL, mx, o));
        rescale(st, mx);
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            st.s += __shfl_xor_sync(ALL, st.s, o);
            st.t += __shfl_xor_sync(ALL, st.t, o);
        }
        if (lane == 0) sh.stats[warp] = st;
        __syncthreads();

        // ---- the alternatives: the warp's list of the keys that reach the bound ----
        uint64_t list = 0;
        if (a.top > 0) {
            thr = sh.bound[0];
#pragma unroll
            for (int w = 1; w < W; ++w) thr = sh.bound[w] < thr ? sh.bound[w] : thr;
            unsigned sel = __ballot_sync(ALL, live && order_of(own_m) >= (uint32_t)(thr >> 32));
            const int mine0 = L0 + warp * 32;                         // lane 0's first vector
            const int per_lane = mine0 < L1 ? (L1 - mine0 + THREADS - 1) / THREADS : 0;
            const int total = __popc(sel) * per_lane;
            for (int i0 = 0; i0 < total; i0 += 32) {
                const int i = i0 + lane;
                const int L = i < total ? mine0 + (int)__fns(sel, 0, i / per_lane + 1) + i % per_lane * THREADS : L1;
                float f[V];
#pragma unroll
                for (int j = 0; j < V; ++j) f[j] = ninf;
                if (L < L1) x.load(L, f);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const uint64_t k = key_of(f[j], (uint32_t)(L * V - x.lead + j));
                    const uint64_t worst = __shfl_sync(ALL, list, a.top - 1);
                    unsigned some = __ballot_sync(ALL, f[j] > ninf && k >= thr && k > worst);
                    for (; some; some &= some - 1) insert32(list, __shfl_sync(ALL, k, __ffs(some) - 1), lane);
                }
            }
            sh.list[warp][lane] = list;
            __syncthreads();
        }

        // ---- join the warps, then the cluster's CTAs ----
        if (warp == 0) {
            Stats all = sh.stats[0];
            for (int w = 1; w < W; ++w) {
                Stats o = sh.stats[w];
                const float top_m = fmaxf(all.m, o.m);
                rescale(all, top_m);
                rescale(o, top_m);
                all.s += o.s;
                all.t += o.t;
                if (a.top > 0) merge32(list, sh.list[w][lane], lane);
            }
            if (CL > 1) {
                asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
                if (a.top > 0)
                    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(remote(&sh.part_list[rank][lane], 0)), "l"(list)
                                 : "memory");
                if (lane == 0) {
                    const uint32_t to = remote(&sh.part_stats[rank], 0);
                    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(all.m) : "memory");
                    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + 4), "f"(all.s) : "memory");
                    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + 8), "f"(all.t) : "memory");
                }
                asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
                if (rank == 0) {
                    all = sh.part_stats[0];
                    list = a.top > 0 ? sh.part_list[0][lane] : 0;
                    for (int c = 1; c < CL; ++c) {
                        Stats o = sh.part_stats[c];
                        const float top_m = fmaxf(all.m, o.m);
                        rescale(all, top_m);
                        rescale(o, top_m);
                        all.s += o.s;
                        all.t += o.t;
                        if (a.top > 0) merge32(list, sh.part_list[c][lane], lane);
                    }
                }
            }
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
        } else if (CL > 1) {
            asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
            asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
        }
        __syncthreads();
    }
}

template <typename T, int THREADS>
cudaError_t launch_rows(const LogprobArgs &a, int64_t m, int64_t v, int CL, cudaStream_t stream)
{
    const int64_t rows = CL > 1 || m < (1 << 24) ? m : (1 << 24);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * CL));
    cfg.blockDim = dim3(THREADS);
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
        // Share a row among CTAs while that leaves two to an SM at most, each with a step of work.
        int CL = 1;
        while (CL < MAX_CL && m * CL * 2 <= 2 * dev.num_sms && v / (CL * 2) >= THREADS * VEC<T>) CL *= 2;
        return launch_rows<T, THREADS>(a, m, v, CL, stream);
    });
}

}  // namespace q8
