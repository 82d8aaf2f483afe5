// rmsnorm.cu -- residual addition, root-mean-square norm and q8_1 quantization in one pass:
//   s = x + r (f32),  y = s * (mean(s^2) + eps)^-1/2 * w,  then the q8_1 blocks of y.
//
// Simple form: one CTA per row; the row is read twice (once for the sum of squares).
#include "launch.h"
#include "q8_1.cuh"
#include "types.cuh"

namespace q8 {
namespace {

constexpr int THREADS = 256;

__device__ __forceinline__ float load_weight(const void *w, int wtype, int64_t i)
{
    if (wtype == Q8ACT_F32) return static_cast<const float *>(w)[i];
    if (wtype == Q8ACT_F16) return to_f32(static_cast<const __half *>(w)[i]);
    return to_f32(static_cast<const __nv_bfloat16 *>(w)[i]);
}

// V consecutive values of the sum x + r as f32.
template <typename T>
__device__ __forceinline__ void load_sum(const T *x, const T *r, int64_t i, float (&v)[VEC<T>])
{
    unpack<T>(*reinterpret_cast<const uint4 *>(x + i), v);
    if (r) {
        float u[VEC<T>];
        unpack<T>(*reinterpret_cast<const uint4 *>(r + i), u);
#pragma unroll
        for (int j = 0; j < VEC<T>; ++j) v[j] = __fadd_rn(v[j], u[j]);
    }
}

template <typename T, bool MMQ>
__global__ void __launch_bounds__(THREADS) rmsnorm_q8_1_kernel(NormArgs a, int64_t m, int k)
{
    constexpr int V = VEC<T>;
    __shared__ float part[THREADS / 32];
    griddep_enter();
    const int chunks = k / V;
    for (int64_t t = blockIdx.x; t < m; t += gridDim.x) {
        const T *x = static_cast<const T *>(a.x) + t * a.ldx;
        const T *r = a.residual ? static_cast<const T *>(a.residual) + t * a.ldr : nullptr;
        float ss = 0.0f;
        for (int c = threadIdx.x; c < chunks; c += THREADS) {
            float v[V];
            load_sum<T>(x, r, (int64_t)c * V, v);
#pragma unroll
            for (int j = 0; j < V; ++j) ss = fmaf(v[j], v[j], ss);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(FULL, ss, o);
        __syncthreads();
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = ss;
        __syncthreads();
        float total = 0.0f;
#pragma unroll
        for (int i = 0; i < THREADS / 32; ++i) total += part[i];
        const float inv = __fdiv_rn(1.0f, sqrtf(total / (float)k + a.eps));
        // chunks is a multiple of 32: a warp is inside the row or past it as a whole
        for (int c = threadIdx.x; c < chunks; c += THREADS) {
            const int64_t i = (int64_t)c * V;
            float v[V];
            load_sum<T>(x, r, i, v);
            if (a.residual_out)
                *reinterpret_cast<uint4 *>(static_cast<T *>(a.residual_out) + t * a.ldro + i) = pack<T>(v);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                v[j] = v[j] * inv;
                if (a.weight) v[j] *= load_weight(a.weight, a.wtype, i + j);
            }
            if (a.y) *reinterpret_cast<uint4 *>(static_cast<T *>(a.y) + t * k + i) = pack<T>(v);
            const BlockQ<V> b = quantize_block<V>(v);
            const bool first = c % (QK / V) == 0;
            if (MMQ) {
                __half *q = reinterpret_cast<__half *>(a.q) + t * k + i;
#pragma unroll
                for (int j = 0; j < V; ++j) q[j] = __float2half_rn(b.t[j]);
                if (first) a.d[(int64_t)(c / (QK / V)) * a.ldm + t] = b.d;
            } else {
                int8_t *q = reinterpret_cast<int8_t *>(a.q) + t * k + i;
#pragma unroll
                for (int j = 0; j < V; ++j) q[j] = (int8_t)b.t[j];
                if (first) a.d[t * (k / QK) + c / (QK / V)] = b.d;
            }
        }
    }
}

}  // namespace

cudaError_t launch_rmsnorm_q8_1(const DeviceInfo &dev, const NormArgs &a, bool mmq, int64_t m, int64_t k, int type,
                                cudaStream_t stream)
{
    return with_type(type, [&](auto t) {
        using T = decltype(t);
        const dim3 grid((unsigned)(m < (1 << 20) ? m : (1 << 20)));
        return mmq ? launch_dependent(rmsnorm_q8_1_kernel<T, true>, grid, THREADS, 0, stream, a, m, (int)k)
                   : launch_dependent(rmsnorm_q8_1_kernel<T, false>, grid, THREADS, 0, stream, a, m, (int)k);
    });
}

}  // namespace q8
