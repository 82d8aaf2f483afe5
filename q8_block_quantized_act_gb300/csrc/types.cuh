// types.cuh -- the element types of activations, residuals, weights of a norm, logits and
// outputs (Q8ACT_F32, Q8ACT_F16, Q8ACT_BF16): 16-byte vectors of them to and from f32.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"

namespace q8 {

template <typename T>
constexpr int VEC = 16 / (int)sizeof(T);   // elements of a 16-byte vector

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

// Round to nearest even, once.
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// A 16-byte vector's elements as f32.
template <typename T>
__device__ __forceinline__ void unpack(uint4 u, float (&v)[VEC<T>])
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
            v[i] = __uint_as_float(w[i]);
        } else if constexpr (std::is_same<T, __half>::value) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        } else {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}

// f32 values rounded to a 16-byte vector of T.
template <typename T>
__device__ __forceinline__ uint4 pack(const float (&v)[VEC<T>])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
            w[i] = __float_as_uint(v[i]);
        } else if constexpr (std::is_same<T, __half>::value) {
            const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        } else {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Host: call f with a value of the element type that `type` names.
template <typename F>
cudaError_t with_type(int type, F &&f)
{
    switch (type) {
    case Q8ACT_F32: return f(float{});
    case Q8ACT_F16: return f(__half{});
    case Q8ACT_BF16: return f(__nv_bfloat16{});
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace q8
