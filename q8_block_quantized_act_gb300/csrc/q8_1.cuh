// q8_1.cuh -- the q8_1 block quantization that the activation quantizers and the fused norm
// share: one block is spread over consecutive lanes, which agree on its amax by shuffles.
#pragma once

#include "common.cuh"

namespace q8 {

constexpr unsigned FULL = 0xffffffffu;

// For normal x (the flushing form is one instruction).
__device__ __forceinline__ float rcp_approx(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
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

// The larger of three magnitudes; NaN wins.
__device__ __forceinline__ float max3_abs_nan(float a, float b, float c)
{
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// V consecutive values of a block whose 32 values are spread over 32 / V lanes.  t: their quants plus
// 1.5 * 2^23, where floats have unit spacing: quant_of is exact (+0 for zero), and the low byte of
// the bits is the quant's two's complement.
constexpr float QUANT_BIAS = 12582912.0f;
template <int V>
struct BlockQ {
    float t[V];
    float d;
};
__device__ __forceinline__ float quant_of(float t) { return __fsub_rn(t, QUANT_BIAS); }
__device__ __forceinline__ uint32_t quant_bytes(const float *t)          // four quants as int8
{
    const uint32_t lo = __byte_perm(__float_as_uint(t[0]), __float_as_uint(t[1]), 0x0040);
    const uint32_t hi = __byte_perm(__float_as_uint(t[2]), __float_as_uint(t[3]), 0x0040);
    return __byte_perm(lo, hi, 0x5410);
}

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
    const float2 rc2 = make_float2(rc, rc), big = make_float2(QUANT_BIAS, QUANT_BIAS);
    float off = 0.0f;                  // one test for the thread: a chain of V would be longer than the work
#pragma unroll
    for (int i = 0; i < V; i += 2) {
        const float2 qa = __fmul2_rn(make_float2(v[i], v[i + 1]), rc2);
        const float2 b = __fadd2_rn(qa, big), n = __fadd2_rn(b, make_float2(-big.x, -big.y));
        const float2 e = __ffma2_rn(n, make_float2(-1.0f, -1.0f), qa);          // qa - n, rounded once
        off = max3_abs_nan(off, e.x, e.y);
        r.t[i] = b.x;
        r.t[i + 1] = b.y;
    }
    if (!(off < 0.4999f)) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (!(fabsf(__fsub_rn(__fmul_rn(v[i], rc), quant_of(r.t[i]))) < 0.4999f))
                r.t[i] = __fadd_rn(quantize_exactly(v[i], r.d), QUANT_BIAS);
    }
    return r;
}

}  // namespace q8
