// q8_1.cuh -- the q8_1 block quantization that the activation quantizers and the fused norm
// share: one block is spread over consecutive lanes, which agree on its amax by shuffles.
#pragma once

#include "common.cuh"

namespace q8 {

constexpr unsigned FULL = 0xffffffffu;

__device__ __forceinline__ float rcp_approx(float x)
{
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// amax / 127 correctly rounded, for amax >= 0: Markstein's correction for a division by a
// known divisor (a quotient q0 = amax * RN(1/127), its exact residual amax - 127 q0 by one FMA,
// and q0 + residual * RN(1/127) by another).  Checked against IEEE division on the host for
// every non-negative binary32 value: all agree except amax = +inf (the residual is then NaN),
// which is selected separately.
__device__ __forceinline__ float div127(float a)
{
    const float c = 1.0f / 127.0f;
    const float q0 = __fmul_rn(a, c);
    const float q1 = __fmaf_rn(__fmaf_rn(-q0, 127.0f, a), c, q0);
    return a == __int_as_float(0x7f800000) ? a : q1;
}

// 1 / d, approximately; 0 for d = 0 (every finite value of the block quantizes to 0), and NaN for a
// subnormal d, whose rounding may leave quotients above 127: all its values take the division.
__device__ __forceinline__ float block_rcp(float d)
{
    return d >= 1.17549435e-38f ? rcp_approx(d) : d == 0.0f ? 0.0f : __int_as_float(0x7fffffff);
}

// The scalar formula for one value of a block with scale d: the IEEE division, round half away.
// Rare, and kept out of the callers' unrolled code.
static __device__ __noinline__ float quantize_exactly(float v, float d)
{
    float t = roundf(__fdiv_rn(v, d));
    if (t > 127.0f) t = 127.0f;
    if (t < -127.0f) t = -127.0f;
    if (!(t == t)) t = 0.0f;           // NaN quantizes to 0
    return __fadd_rn(t, 0.0f);         // -0 -> +0
}

// V consecutive values of a block whose 32 values are spread over 32 / V lanes: their quants as
// integer-valued floats (+0 for zero).
template <int V>
struct BlockQ {
    float t[V];
    float d;
};

// For a value whose approximate quotient qa = v * block_rcp(d) lies farther than 1e-4 from every
// half-integer, its nearest integer is round-half-away(fl(v / d)): qa differs from v / d by under
// 4e-5 (|v / d| <= 127; the reciprocal's relative error is at most 2^-23, the product's 2^-24) and
// fl(v / d) from v / d by under 8e-6, so all three round to the same integer, at most 127, and no tie
// is involved.  The test |qa - t| < 0.4999 holds for exactly those values; a thread with one that
// fails it (near a half-integer, or qa not finite) takes the scalar formula for that one.  The nearest integer
// comes from adding and subtracting 1.5 * 2^23 (unit spacing there), two values an instruction.
template <int V>
__device__ __forceinline__ BlockQ<V> quantize_block(const float (&v)[V])
{
    float a = 0.0f;                    // a block of NaNs behaves like the scalar loop's "a > amax"
#pragma unroll
    for (int i = 0; i < V; ++i) a = fmaxf(a, fabsf(v[i]));
#pragma unroll
    for (int o = 1; o < 32 / V; o <<= 1) a = fmaxf(a, __shfl_xor_sync(FULL, a, o));
    BlockQ<V> r;
    r.d = div127(a);
    const float rc = block_rcp(r.d);
    const float2 rc2 = make_float2(rc, rc), big = make_float2(12582912.0f, 12582912.0f);
    bool fine = true;
#pragma unroll
    for (int i = 0; i < V; i += 2) {
        const float2 qa = __fmul2_rn(make_float2(v[i], v[i + 1]), rc2);
        const float2 t = __fadd2_rn(__fadd2_rn(qa, big), make_float2(-big.x, -big.y));
        const float2 e = __ffma2_rn(t, make_float2(-1.0f, -1.0f), qa);          // qa - t, rounded once
        fine = fine && fabsf(e.x) < 0.4999f && fabsf(e.y) < 0.4999f;
        r.t[i] = t.x;
        r.t[i + 1] = t.y;
    }
    if (!fine) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (!(fabsf(__fsub_rn(__fmul_rn(v[i], rc), r.t[i])) < 0.4999f)) r.t[i] = quantize_exactly(v[i], r.d);
    }
    return r;
}

// An integer-valued float t, |t| <= 127, as its int8 byte: the bits of t + 1.5 * 2^23 are
// those of 1.5 * 2^23 plus t (unit spacing there), so the low byte is t's two's complement.
__device__ __forceinline__ uint32_t byte_of(float t)
{
    return (uint32_t)__float_as_int(__fadd_rn(t, 12582912.0f)) & 0xFFu;
}

}  // namespace q8
