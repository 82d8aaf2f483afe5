// mxfp4.cuh -- the MXFP4 block format: 32 values share a power-of-two scale (one e8m0 byte b,
// 2^(b - 127), b = 255 for a block that holds a NaN or an infinity), each value is an e2m1 code
// (sign, magnitude 0 0.5 1 1.5 2 3 4 6).  Codes: two to a byte, the even one in the low nibble,
// rows of k / 2 bytes.  Scales: tiles of 128 rows x 128 values (4 blocks), 512 bytes each, the
// order that the block-scaled tensor-core product copies into tensor memory as it stands.
#pragma once

#include "types.cuh"

namespace q8 {

constexpr int MX_TILE_ROWS = 128;
constexpr int MX_TILE_K = 128;
constexpr int MX_TILE_BYTES = 512;

// Offset of the scale byte of row r, block b.
__host__ __device__ __forceinline__ int64_t mx_scale_at(int64_t r, int b, int ktiles)
{
    return ((r >> 7) * ktiles + (b >> 2)) * MX_TILE_BYTES + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (b & 3);
}

// 2^(b - 127) for a scale byte (b = 255: NaN); b = 0 is the subnormal 2^-127.
__device__ __forceinline__ float mx_scale(uint32_t b)
{
    return __uint_as_float(b == 255u ? 0x7fffffffu : (b == 0u ? 0x00400000u : b << 23));
}

// The scale byte of a block from the largest of its values' absolute bits:
// E = floor(log2 amax) - 2 (the largest code's exponent), clamped to 2^-127 from below.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits)
{
    if (amax_bits >= 0x7f800000u) return 255u;
    const uint32_t e = amax_bits >> 23;
    return e > 2u ? e - 2u : 0u;
}

// 2^(127 - b), the exact factor that brings a block's values onto the code's grid (b <= 252).
__device__ __forceinline__ float mx_inverse(uint32_t b) { return __uint_as_float((254u - b) << 23); }

// Eight values already scaled by mx_inverse to eight codes: nearest, ties to the even code,
// saturating at 6.
__device__ __forceinline__ uint32_t mx_codes8(const float (&v)[8])
{
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// The largest absolute bits of 8 values, as those of an f32 (infinities and NaN above all others):
// in 16-bit types the comparison takes two values an instruction.
template <typename T>
__device__ __forceinline__ uint32_t largest_bits(const uint4 (&u)[sizeof(T) / 2])
{
    if constexpr (sizeof(T) == 4) {
        const uint32_t w[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w};
        uint32_t a = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) a = max(a, w[i] & 0x7fffffffu);
        return a;
    } else {
        using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
        const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
        T2 q = __habs2(*reinterpret_cast<const T2 *>(&w[0]));
#pragma unroll
        for (int i = 1; i < 4; ++i) q = __hmax2_nan(q, __habs2(*reinterpret_cast<const T2 *>(&w[i])));
        const uint32_t p = *reinterpret_cast<const uint32_t *>(&q);
        const uint32_t a = max(p & 0xffffu, p >> 16);          // NaN is above infinity
        if constexpr (std::is_same<T, __half>::value) return __float_as_uint(half_bits_to_float(a));
        else return a << 16;
    }
}

// A warp's 256 consecutive values, 8 a lane: this lane's codes, and in every 16th lane the four scale
// bytes of its 128 values (a block with a NaN or an infinity: byte 255, codes 0).
struct MxChunk {
    uint32_t codes, scales;
};
template <typename T>
__device__ __forceinline__ MxChunk mx_quantize8(const uint4 (&in)[sizeof(T) / 2])
{
    uint32_t a = largest_bits<T>(in);
    a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
    a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
    const uint32_t b = mx_scale_byte(a);
    float v[8];
    if constexpr (sizeof(T) == 4) {
        float lo[4], hi[4];
        unpack<T>(in[0], lo);
        unpack<T>(in[1], hi);
#pragma unroll
        for (int i = 0; i < 4; ++i) { v[i] = lo[i]; v[4 + i] = hi[i]; }
    } else {
        unpack<T>(in[0], v);
    }
    const float inv = b == 255u ? 0.0f : mx_inverse(b);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const float2 p = __fmul2_rn(make_float2(v[i], v[i + 1]), make_float2(inv, inv));
        v[i] = p.x;
        v[i + 1] = p.y;
    }
    const uint32_t codes = b == 255u ? 0u : mx_codes8(v);
    uint32_t word = b | (__shfl_down_sync(0xffffffffu, b, 4) << 8);
    word |= __shfl_down_sync(0xffffffffu, word, 8) << 16;
    return {codes, word};
}

}  // namespace q8
