// mxfp4.cu -- MXFP4 quantization (activations and weights), its mirror, and the tiling of
// row-major scales.  Elementwise passes bound by memory: at 20480 x 4096 bf16 the quantizer takes
// 32.7 us and the mirror 32.6 (6.5 TB/s each, 0.96 of a copy).  Scaling by a power of two is exact,
// so the conversion to a code is the only rounding of the quantizer, and the mirror's to its type
// the only one there.
#include "launch.h"
#include "mxfp4.cuh"
#include "types.cuh"

namespace q8 {
namespace {

// A thread has 8 consecutive values of each of ROWS rows, 4 lanes a block; the four scale bytes of
// 128 values leave as one word.  ROWS = 4: the rows are 32 apart, so that their words are neighbours
// in the scale tile and leave as one 16-byte store (four scattered words cost 9 of 41 us at
// 20480 x 4096).  Rows m .. 128 ceil(m / 128) - 1 get zero scale bytes, so that the whole scale array
// is defined.
template <typename T, int ROWS>
__global__ void __launch_bounds__(256) quantize_mxfp4_kernel(const T *__restrict__ x, int64_t ldx,
                                                             uint32_t *__restrict__ codes,
                                                             uint8_t *__restrict__ scales, int64_t m, int k)
{
    static_assert(ROWS == 1 || ROWS == 4, "rows of a thread");
    constexpr int APART = 32;
    griddep_enter();
    const int chunks = k / 8;
    const int c = blockIdx.x * blockDim.x + threadIdx.x;
    if (c >= chunks) return;          // k / 8 is a multiple of 32: warps are whole
    const int64_t padded = (m + MX_TILE_ROWS - 1) / MX_TILE_ROWS * MX_TILE_ROWS;
    for (int64_t g = blockIdx.y; g * ROWS < padded; g += gridDim.y) {
        const int64_t r0 = ROWS == 1 ? g : g / APART * MX_TILE_ROWS + g % APART;
        uint4 in[ROWS][sizeof(T) / 2];
#pragma unroll
        for (int j = 0; j < ROWS; ++j)
#pragma unroll
            for (int h = 0; h < (int)sizeof(T) / 2; ++h)
                in[j][h] = r0 + j * APART < m ? __ldg(reinterpret_cast<const uint4 *>(x + (r0 + j * APART) * ldx + (int64_t)c * 8) + h)
                                              : make_uint4(0, 0, 0, 0);
        uint32_t words[ROWS];
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            const MxChunk q = mx_quantize8<T>(in[j]);
            if (r0 + j * APART < m) codes[(r0 + j * APART) * chunks + c] = q.codes;
            words[j] = r0 + j * APART < m ? q.scales : 0u;
        }
        if ((c & 15) == 0) {
            uint8_t *to = scales + mx_scale_at(r0, c >> 2, k / MX_TILE_K);
            if constexpr (ROWS == 4) *reinterpret_cast<uint4 *>(to) = make_uint4(words[0], words[1], words[2], words[3]);
            else *reinterpret_cast<uint32_t *>(to) = words[0];
        }
    }
}

// The values of V = 8 or 4 codes (two at a time through binary16, which holds them exactly).
template <int V>
__device__ __forceinline__ void mx_values(uint32_t w, float (&v)[V])
{
    uint32_t h[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

// A thread makes 16 bytes of each of ROWS rows: 8 values, or 4 of f32 (8 of f32 would leave in two
// stores 32 bytes apart: 42.4 us instead of 29.6 at 10240 x 4096).
template <typename T, int ROWS>
__global__ void __launch_bounds__(256) dequant_mxfp4_kernel(const uint8_t *__restrict__ codes,
                                                            const uint8_t *__restrict__ scales, T *__restrict__ y,
                                                            int64_t m, int k)
{
    constexpr int V = VEC<T>;
    using Codes = typename std::conditional<V == 8, uint32_t, uint16_t>::type;
    griddep_enter();
    const int chunks = k / V;
    const int c = blockIdx.x * blockDim.x + threadIdx.x;
    if (c >= chunks) return;
    for (int64_t r0 = (int64_t)blockIdx.y * ROWS; r0 < m; r0 += (int64_t)gridDim.y * ROWS) {
        uint32_t w[ROWS], b[ROWS];
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            w[j] = r0 + j < m ? reinterpret_cast<const Codes *>(codes)[(r0 + j) * chunks + c] : 0u;
            b[j] = r0 + j < m ? scales[mx_scale_at(r0 + j, c / (QK / V), k / MX_TILE_K)] : 0u;
        }
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            if (r0 + j >= m) break;
            const float s = mx_scale(b[j]);
            float v[V];
            mx_values<V>(w[j], v);
#pragma unroll
            for (int i = 0; i < V; i += 2) {
                const float2 p = __fmul2_rn(make_float2(v[i], v[i + 1]), make_float2(s, s));
                v[i] = p.x;
                v[i + 1] = p.y;
            }
            *reinterpret_cast<uint4 *>(y + (r0 + j) * k + (int64_t)c * V) = pack<T>(v);
        }
    }
}

// Load-time: one byte a thread (0.3 % of the weights' values).
__global__ void __launch_bounds__(256) tile_mxfp4_scales_kernel(const uint8_t *__restrict__ src,
                                                                uint8_t *__restrict__ dst, int64_t m, int kb)
{
    griddep_enter();
    const int64_t padded = (m + MX_TILE_ROWS - 1) / MX_TILE_ROWS * MX_TILE_ROWS;
    const int64_t stride = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < padded * kb; i += stride) {
        const int64_t r = i / kb;
        const int b = (int)(i % kb);
        dst[mx_scale_at(r, b, kb / 4)] = r < m ? src[i] : 0;
    }
}

// CTAs of at most 256 threads that share a row's chunks (a multiple of 32) evenly.
struct RowGrid {
    dim3 grid;
    int threads;
};
RowGrid grid_rows(int64_t rows, int64_t chunks, int each)
{
    const int64_t groups = (rows + each - 1) / each, ctas = (chunks + 255) / 256;
    return {dim3((unsigned)ctas, (unsigned)(groups < 65535 ? groups : 65535)),
            (int)(((chunks + ctas - 1) / ctas + 31) / 32 * 32)};
}

}  // namespace

cudaError_t launch_quantize_mxfp4(const DeviceInfo &dev, const void *x, int64_t ldx, int type, uint8_t *codes,
                                  uint8_t *scales, int64_t m, int64_t k, cudaStream_t stream)
{
    return with_type(type, [&](auto t) {
        using T = decltype(t);
        const int64_t padded = (m + MX_TILE_ROWS - 1) / MX_TILE_ROWS * MX_TILE_ROWS;
        auto go = [&](auto kern, int each) {
            const RowGrid g = grid_rows(padded, k / 8, each);
            return launch_dependent(kern, g.grid, g.threads, 0, stream, static_cast<const T *>(x), ldx,
                                    reinterpret_cast<uint32_t *>(codes), scales, m, (int)k);
        };
        // Four rows a thread (more bytes under way) from so many chunks an SM on; below, latency counts.
        // One row and four: 256 x 4096 f32 2.3 and 2.7 us, 8192 x 4096 f32 24.2 and 23.5; 1024 x 4096 bf16
        // 3.8 and 4.1, 2048 x 4096 bf16 6.4 and 5.4, 8192 x 4096 bf16 20.8 and 14.1.
        const int64_t from = sizeof(T) == 4 ? 8192 : 4000;
        return m * (k / 8) >= dev.num_sms * from ? go(quantize_mxfp4_kernel<T, 4>, 4) : go(quantize_mxfp4_kernel<T, 1>, 1);
    });
}

cudaError_t launch_dequant_mxfp4(const DeviceInfo &dev, const uint8_t *codes, const uint8_t *scales, void *y, int type,
                                 int64_t m, int64_t k, cudaStream_t stream)
{
    return with_type(type, [&](auto t) {
        using T = decltype(t);
        auto go = [&](auto kern, int each) {
            const RowGrid g = grid_rows(m, k / VEC<T>, each);
            return launch_dependent(kern, g.grid, g.threads, 0, stream, codes, scales, static_cast<T *>(y), m, (int)k);
        };
        // One row a thread and four: 512 x 1024 bf16 1.6 and 1.8 us, 1024 x 4096 bf16 3.8 and 3.3,
        // 8192 x 4096 bf16 20.8 and 13.5, 1024 x 4096 f32 5.7 and 4.6.
        return m * (k / VEC<T>) >= (int64_t)dev.num_sms * 800 ? go(dequant_mxfp4_kernel<T, 4>, 4) : go(dequant_mxfp4_kernel<T, 1>, 1);
    });
}

cudaError_t launch_tile_mxfp4_scales(const DeviceInfo &dev, const uint8_t *src, uint8_t *dst, int64_t m, int64_t k,
                                     cudaStream_t stream)
{
    const int64_t total = (m + MX_TILE_ROWS - 1) / MX_TILE_ROWS * MX_TILE_ROWS * (k / QK);
    const int64_t want = (total + 255) / 256, cap = (int64_t)dev.num_sms * 8;
    return launch_dependent(tile_mxfp4_scales_kernel, dim3((unsigned)(want < cap ? want : cap)), 256, 0, stream, src,
                            dst, m, (int)(k / QK));
}

}  // namespace q8
