// rmsnorm.cu -- residual addition, root-mean-square norm and q8_1 quantization in one pass:
//   s = x + r (f32),  y = s * (mean(s^2) + eps)^-1/2 * w,  then the q8_1 blocks of y.
//
// Bound by memory: x, the residual in, the residual, the quants and scales out.  The row stays in
// registers between the sum of squares and the quantization, so each is moved once.  4093 x 8192
// f16: 39.4 us with a residual to int8 (6.1 TB/s, 0.90 of a copy), the norm alone 41.9 (0.94).  Without
// a residual 29.4 to int8, 30.7 to binary16 (0.52 and 0.66 of a copy): the instructions (21 a value)
// would take 18 us and the bytes 20, but each row's loads, barrier and shuffles follow one another and 64
// registers leave four rows an SM to overlap them (issue slots 62 % busy, no pipe above 31 %; most
// waiting is for loads, then for fixed latencies).  All
// arithmetic is f32; the residual is rounded once to its type, y once, the norm itself not at all
// before the quantization.
#include "launch.h"
#include "q8_1.cuh"
#include "types.cuh"

namespace q8 {
namespace {

// V consecutive weights as f32.
template <int V, typename W>
__device__ __forceinline__ void load_weights(const W *w, float (&f)[V])
{
    if constexpr (V == VEC<W>) {
        unpack<W>(__ldg(reinterpret_cast<const uint4 *>(w)), f);
    } else if constexpr (V > VEC<W>) {             // 8 of 4 bytes
        float g[4];
        unpack<W>(__ldg(reinterpret_cast<const uint4 *>(w)), g);
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = g[j];
        unpack<W>(__ldg(reinterpret_cast<const uint4 *>(w) + 1), g);
#pragma unroll
        for (int j = 0; j < 4; ++j) f[4 + j] = g[j];
    } else {                                       // 4 of 2 bytes
        const uint2 u = __ldg(reinterpret_cast<const uint2 *>(w));
        float g[8];
        unpack<W>(make_uint4(u.x, u.y, 0, 0), g);
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = g[j];
    }
}

// Two products an instruction.
template <int V>
__device__ __forceinline__ void times(float (&v)[V], const float (&w)[V])
{
#pragma unroll
    for (int j = 0; j < V; j += 2) {
        const float2 p = __fmul2_rn(make_float2(v[j], v[j + 1]), make_float2(w[j], w[j + 1]));
        v[j] = p.x;
        v[j + 1] = p.y;
    }
}
template <int V>
__device__ __forceinline__ void times(float (&v)[V], float f)
{
#pragma unroll
    for (int j = 0; j < V; j += 2) {
        const float2 p = __fmul2_rn(make_float2(v[j], v[j + 1]), make_float2(f, f));
        v[j] = p.x;
        v[j + 1] = p.y;
    }
}

template <int V>
__device__ __forceinline__ void weigh(const NormArgs &a, int64_t i, float (&v)[V])
{
    float w[V];
    if (a.wtype == Q8ACT_F32) load_weights<V>(static_cast<const float *>(a.weight) + i, w);
    else if (a.wtype == Q8ACT_F16) load_weights<V>(static_cast<const __half *>(a.weight) + i, w);
    else load_weights<V>(static_cast<const __nv_bfloat16 *>(a.weight) + i, w);
    times<V>(v, w);
}

template <typename T>
__device__ __forceinline__ bool is_type(int type)
{
    return type == (sizeof(T) == 4 ? Q8ACT_F32 : std::is_same<T, __half>::value ? Q8ACT_F16 : Q8ACT_BF16);
}

// The quants and scale of chunk c of row t: V values of the block that starts at a multiple of
// 32 / V lanes.
template <typename T, bool MMQ>
__device__ __forceinline__ void store_block(const NormArgs &a, int64_t t, int k, int c, const float (&v)[VEC<T>])
{
    constexpr int V = VEC<T>;
    const int64_t i = t * k + (int64_t)c * V;
    if (a.y) *reinterpret_cast<uint4 *>(static_cast<T *>(a.y) + i) = pack<T>(v);
    if (!a.q) return;
    const BlockQ<V> b = quantize_block<V>(v);
    const bool first = c % (QK / V) == 0;
    if constexpr (MMQ) {
        uint32_t w[V / 2];                         // small integers: exact in binary16
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
            const __half2 h = __floats2half2_rn(quant_of(b.t[2 * j]), quant_of(b.t[2 * j + 1]));
            w[j] = *reinterpret_cast<const uint32_t *>(&h);
        }
        uint16_t *q = static_cast<uint16_t *>(a.q) + i;
        if constexpr (V == 8) *reinterpret_cast<uint4 *>(q) = make_uint4(w[0], w[1], w[2], w[3]);
        else *reinterpret_cast<uint2 *>(q) = make_uint2(w[0], w[1]);
        if (first) a.d[(int64_t)(c / (QK / V)) * a.ldm + t] = b.d;
    } else {
        int8_t *q = static_cast<int8_t *>(a.q) + i;
        if constexpr (V == 8) *reinterpret_cast<uint2 *>(q) = make_uint2(quant_bytes(b.t), quant_bytes(b.t + 4));
        else *reinterpret_cast<uint32_t *>(q) = quant_bytes(b.t);
        if (first) a.d[t * (k / QK) + c / (QK / V)] = b.d;
    }
}

// The CTA's sum, the same in every thread.
__device__ __forceinline__ float cta_sum(float s, float *part)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(FULL, s, o);
    const int warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
    __syncthreads();
    float v = (int)(threadIdx.x & 31) < warps ? part[threadIdx.x & 31] : 0.0f;
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
    return v;
}

template <typename T>
__device__ __forceinline__ void add_residual(uint4 x, uint4 r, bool add, float (&v)[VEC<T>])
{
    unpack<T>(x, v);
    if (add) {
        float u[VEC<T>];
        unpack<T>(r, u);
#pragma unroll
        for (int j = 0; j < VEC<T>; ++j) v[j] = __fadd_rn(v[j], u[j]);
    }
}

// A CTA per row, CH 16-byte chunks a thread.  chunks = k / V is a multiple of 32, so a warp's chunk
// is inside the row for all of its lanes or for none, as the block's shuffles need.  Weights of x's
// type are loaded beside the row, before the barrier.
template <typename T, bool MMQ, int CH, int MAX_THREADS>
__global__ void __launch_bounds__(MAX_THREADS, 1024 / MAX_THREADS) rmsnorm_row_kernel(NormArgs a, int k)
{
    constexpr int V = VEC<T>;
    __shared__ float part[32];
    griddep_enter();
    const int chunks = k / V;
    const int64_t t = blockIdx.x;
    const uint4 *x = reinterpret_cast<const uint4 *>(static_cast<const T *>(a.x) + t * a.ldx);
    const uint4 *r = reinterpret_cast<const uint4 *>(static_cast<const T *>(a.residual) + t * a.ldr);
    const bool early = a.weight && is_type<T>(a.wtype);
    uint4 xv[CH], rv[CH], wv[CH];
    if ((int)blockDim.x * CH == chunks) {                 // no thread is without a chunk
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            xv[i] = x[threadIdx.x + i * blockDim.x];
            if (a.residual) rv[i] = r[threadIdx.x + i * blockDim.x];
        }
    } else {
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            xv[i] = c < chunks ? x[c] : make_uint4(0, 0, 0, 0);
            if (a.residual) rv[i] = c < chunks ? r[c] : make_uint4(0, 0, 0, 0);
        }
    }
    if (early)
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c < chunks) wv[i] = __ldg(static_cast<const uint4 *>(a.weight) + c);
        }
    float v[CH][V];
    float2 ss = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        add_residual<T>(xv[i], rv[i], a.residual != nullptr, v[i]);
#pragma unroll
        for (int j = 0; j < V; j += 2) {
            const float2 p = make_float2(v[i][j], v[i][j + 1]);
            ss = __ffma2_rn(p, p, ss);
        }
    }
    if (a.residual_out) {
        T *out = static_cast<T *>(a.residual_out) + t * a.ldro;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c < chunks) *reinterpret_cast<uint4 *>(out + (int64_t)c * V) = pack<T>(v[i]);
        }
    }
    const float inv = rsqrtf(cta_sum(ss.x + ss.y, part) * a.inv_k + a.eps);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        times<V>(v[i], inv);
        if (early) {
            float w[V];
            unpack<T>(wv[i], w);
            times<V>(v[i], w);
        } else if (a.weight && c < chunks) {
            weigh<V>(a, (int64_t)c * V, v[i]);
        }
        if (c < chunks) store_block<T, MMQ>(a, t, k, c, v[i]);
    }
}

// Rows too long for registers: read twice, the second time from L2 at best, with a chunk a thread under way
// (4093 x 20480 f32: 245 us with a residual and no quants, 0.81 of a copy; 161 to int8 without, 0.39).
template <typename T, bool MMQ>
__global__ void __launch_bounds__(1024) rmsnorm_long_kernel(NormArgs a, int k)
{
    constexpr int V = VEC<T>;
    __shared__ float part[32];
    griddep_enter();
    const int chunks = k / V;
    const int64_t t = blockIdx.x;
    const uint4 *x = reinterpret_cast<const uint4 *>(static_cast<const T *>(a.x) + t * a.ldx);
    const uint4 *r = a.residual ? reinterpret_cast<const uint4 *>(static_cast<const T *>(a.residual) + t * a.ldr) : nullptr;
    float ss = 0.0f;
    for (int c = threadIdx.x; c < chunks; c += blockDim.x) {
        float v[V];
        add_residual<T>(x[c], r ? r[c] : make_uint4(0, 0, 0, 0), r != nullptr, v);
#pragma unroll
        for (int j = 0; j < V; ++j) ss = fmaf(v[j], v[j], ss);
    }
    const float inv = rsqrtf(cta_sum(ss, part) * a.inv_k + a.eps);
    for (int c = threadIdx.x; c < chunks; c += blockDim.x) {
        float v[V];
        add_residual<T>(x[c], r ? r[c] : make_uint4(0, 0, 0, 0), r != nullptr, v);
        if (a.residual_out)
            *reinterpret_cast<uint4 *>(static_cast<T *>(a.residual_out) + t * a.ldro + (int64_t)c * V) = pack<T>(v);
        times<V>(v, inv);
        if (a.weight) weigh<V>(a, (int64_t)c * V, v);
        store_block<T, MMQ>(a, t, k, c, v);
    }
}

template <typename T, bool MMQ>
cudaError_t launch_rows(const DeviceInfo &dev, const NormArgs &a, int64_t m, int64_t k, cudaStream_t stream)
{
    const int chunks = (int)(k / VEC<T>);                  // a multiple of 32
    const dim3 grid((unsigned)m);
    // A row to an SM at most: every thread that a CTA can have, one chunk each if that is enough
    // (latency).  More: small CTAs with up to four chunks a thread, so that several rows are under way
    // on an SM and one row's barrier leaves the others working (1024, 512, 256 threads: 64 x 8192 bf16
    // 3.1, 3.4, 4.3 us; 256 x 8192 bf16 5.9, 4.6, 5.6; 304 x 4096 f32 3.9, 4.4; 512 x 4096 f32 5.7, 5.4,
    // 4.8; 4093 x 8192 f32 67, 43, too long for 256; 8192 x 8192 bf16 137, 85, 67; 256, 128, 64 threads:
    // 1024 x 4096 bf16 7.2, 7.7, 18; 8192 x 1024 f32 13.5, 11.3, 11.3).
    const int sms = dev.num_sms;
    const int about = m <= sms || (m <= 2 * sms && VEC<T> == 4 && chunks <= 1024) ? 1024
                      : m <= 2 * sms ? 512 : m <= 20 * sms ? 256 : 128;
    int share = (chunks + about / 2) / about;              // chunks a thread, to the nearest
    share = share < 1 ? 1 : share > 4 ? 4 : share;
    int threads = ((chunks + share - 1) / share + 31) / 32 * 32;
    if (threads > 1024) threads = 1024;
    const int each = (chunks + threads - 1) / threads;
    auto go = [&](auto kern) { return launch_dependent(kern, grid, threads, 0, stream, a, (int)k); };
    if (each == 1) return go(rmsnorm_row_kernel<T, MMQ, 1, 1024>);
    if (each == 2) return go(rmsnorm_row_kernel<T, MMQ, 2, 1024>);
    if (each <= 4) return threads <= 256 ? go(rmsnorm_row_kernel<T, MMQ, 4, 256>) : go(rmsnorm_row_kernel<T, MMQ, 4, 1024>);
    return launch_dependent(rmsnorm_long_kernel<T, MMQ>, grid, 1024, 0, stream, a, (int)k);
}

}  // namespace

cudaError_t launch_rmsnorm_q8_1(const DeviceInfo &dev, const NormArgs &a, bool mmq, int64_t m, int64_t k, int type,
                                cudaStream_t stream)
{
    return with_type(type, [&](auto t) {
        using T = decltype(t);
        return mmq ? launch_rows<T, true>(dev, a, m, k, stream) : launch_rows<T, false>(dev, a, m, k, stream);
    });
}

}  // namespace q8
