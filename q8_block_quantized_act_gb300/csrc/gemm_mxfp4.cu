// gemm_mxfp4.cu -- the product of two MXFP4 matrices:
//   y[t][r] = sum_b 2^(Ew[r][b] + Ex[t][b]) sum_{i<32} w[r][32b+i] x[t][32b+i],  f32 accumulation.
//
// Simple form: a CTA computes 64 weight rows x 16 tokens, decoding one 32-wide block of both
// operands to f32 in shared memory at a time.
#include "launch.h"
#include "mxfp4.cuh"
#include "types.cuh"

namespace q8 {
namespace {

constexpr int TR = 64, TT = 16;

template <typename T>
__global__ void __launch_bounds__(256) gemm_mxfp4_kernel(const uint8_t *__restrict__ w, const uint8_t *__restrict__ wsc,
                                                         const uint8_t *__restrict__ x, const uint8_t *__restrict__ xsc,
                                                         T *__restrict__ y, int64_t m, int64_t n, int k)
{
    __shared__ float sw[32][TR + 1];
    __shared__ float sx[32][TT + 1];
    griddep_enter();
    const int64_t r0 = (int64_t)blockIdx.x * TR;
    const int tr = threadIdx.x & 63, tq = threadIdx.x >> 6;
    for (int64_t t0 = (int64_t)blockIdx.y * TT; t0 < m; t0 += (int64_t)gridDim.y * TT) {
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
        for (int b = 0; b < k / QK; ++b) {
            __syncthreads();
            for (int i = threadIdx.x; i < TR * 16; i += 256) {
                const int64_t r = r0 + i / 16;
                const uint32_t c = r < n ? w[r * (k / 2) + b * 16 + i % 16] : 0u;
                const float s = r < n ? 0.5f * mx_scale(wsc[mx_scale_at(r, b, k / MX_TILE_K)]) : 0.0f;
                sw[2 * (i % 16)][i / 16] = s * (float)mx_twice(c);
                sw[2 * (i % 16) + 1][i / 16] = s * (float)mx_twice(c >> 4);
            }
            {
                const int i = threadIdx.x;
                const int64_t t = t0 + i / 16;
                const uint32_t c = t < m ? x[t * (k / 2) + b * 16 + i % 16] : 0u;
                const float s = t < m ? 0.5f * mx_scale(xsc[mx_scale_at(t, b, k / MX_TILE_K)]) : 0.0f;
                sx[2 * (i % 16)][i / 16] = s * (float)mx_twice(c);
                sx[2 * (i % 16) + 1][i / 16] = s * (float)mx_twice(c >> 4);
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 32; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[j] = fmaf(sw[i][tr], sx[i][4 * tq + j], acc[j]);
        }
        for (int j = 0; j < 4; ++j) {
            const int64_t t = t0 + 4 * tq + j;
            if (r0 + tr < n && t < m) y[t * n + r0 + tr] = from_f32<T>(acc[j]);
        }
    }
}

}  // namespace

cudaError_t launch_gemm_mxfp4(const DeviceInfo &dev, const uint8_t *w, const uint8_t *wsc, const uint8_t *x,
                              const uint8_t *xsc, void *y, int type, int64_t m, int64_t n, int64_t k,
                              cudaStream_t stream)
{
    return with_type(type, [&](auto t) {
        using T = decltype(t);
        const int64_t gy = (m + TT - 1) / TT;
        return launch_dependent(gemm_mxfp4_kernel<T>, dim3((unsigned)((n + TR - 1) / TR), (unsigned)(gy < 65535 ? gy : 65535)),
                                256, 0, stream, w, wsc, x, xsc, static_cast<T *>(y), m, n, (int)k);
    });
}

}  // namespace q8
