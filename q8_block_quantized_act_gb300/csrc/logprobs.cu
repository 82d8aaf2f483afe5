// logprobs.cu -- for each row of logits: the log probability of a given token, the entropy of
// the softmax, and the most likely tokens with their log probabilities.
//   mx = max x,  S = sum e^(x - mx),  T = sum (x - mx) e^(x - mx)
//   log p(i) = x_i - mx - log S,      H = log S - T / S
// A row whose logits are all -inf has no distribution: log probabilities -inf, entropy 0, no
// alternatives (id -1).  A row with a NaN or +inf: NaN everywhere, ids -1.
//
// Simple form: one CTA per row, three kinds of passes over the row (maximum, sums, and one for
// each alternative).
#include "launch.h"
#include "types.cuh"

namespace q8 {
namespace {

constexpr int THREADS = 512;

// Larger logits and, among equal ones, lower indexes have larger keys; 0 is below every key.
__device__ __forceinline__ uint64_t key_of(float x, uint32_t i)
{
    const uint32_t b = __float_as_uint(x == 0.0f ? 0.0f : x);      // -0 and +0 are equal
    const uint32_t o = (b & 0x80000000u) ? ~b : b | 0x80000000u;
    return ((uint64_t)o << 32) | (uint32_t)~i;
}

__device__ __forceinline__ float value_of(uint64_t key)
{
    const uint32_t o = (uint32_t)(key >> 32);
    return __uint_as_float((o & 0x80000000u) ? o & 0x7fffffffu : ~o);
}

template <typename T>
__global__ void __launch_bounds__(THREADS) logprobs_kernel(LogprobArgs a, int64_t m, int v)
{
    __shared__ uint64_t keys[THREADS / 32];
    __shared__ float sums[2][THREADS / 32];
    __shared__ uint64_t best;
    griddep_enter();
    const float ninf = __int_as_float(0xff800000), nan = __int_as_float(0x7fffffff);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int64_t row = blockIdx.x; row < m; row += gridDim.x) {
        const T *x = static_cast<const T *>(a.logits) + row * a.ld;
        uint64_t below = ~0ull;
        float mx = ninf, lse = 0.0f;
        bool bad = false, empty = false;
        for (int j = 0; j <= a.top; ++j) {
            // j = 0: the row's maximum and whether it has a NaN; then the j-th alternative
            uint64_t k = 0;
            bool nans = false;
            for (int i = threadIdx.x; i < v; i += THREADS) {
                const float f = to_f32(x[i]);
                nans |= !(f < __int_as_float(0x7f800000));
                const uint64_t c = key_of(f, (uint32_t)i);
                if (c < below && c > k && f > ninf) k = c;
            }
            for (int o = 16; o; o >>= 1) {
                const uint64_t other = __shfl_xor_sync(0xffffffffu, k, o);
                if (other > k) k = other;
            }
            const bool any = __syncthreads_or(nans);
            if (lane == 0) keys[warp] = k;
            __syncthreads();
            if (threadIdx.x == 0) {
                for (int w = 1; w < THREADS / 32; ++w)
                    if (keys[w] > k) k = keys[w];
                best = k;
            }
            __syncthreads();
            k = best;
            if (j == 0) {
                bad = any;
                empty = k == 0;
                mx = empty ? 0.0f : value_of(k);
                float s = 0.0f, ts = 0.0f;
                for (int i = threadIdx.x; i < v; i += THREADS) {
                    const float z = to_f32(x[i]) - mx, e = expf(z);
                    s += e;
                    if (e > 0.0f) ts = fmaf(z, e, ts);
                }
                for (int o = 16; o; o >>= 1) {
                    s += __shfl_xor_sync(0xffffffffu, s, o);
                    ts += __shfl_xor_sync(0xffffffffu, ts, o);
                }
                if (lane == 0) { sums[0][warp] = s; sums[1][warp] = ts; }
                __syncthreads();
                s = ts = 0.0f;
                for (int w = 0; w < THREADS / 32; ++w) { s += sums[0][w]; ts += sums[1][w]; }
                lse = empty ? 0.0f : logf(s);
                if (threadIdx.x == 0) {
                    if (a.entropy) a.entropy[row] = bad ? nan : empty ? 0.0f : lse - ts / s;
                    if (a.logprob) {
                        const int32_t t = a.tokens[row];
                        a.logprob[row] = t < 0 ? 0.0f : t >= v || bad ? nan : (to_f32(x[t]) - mx) - lse;
                    }
                }
            } else {
                if (threadIdx.x == 0) {
                    a.top_ids[row * a.top + j - 1] = bad || k == 0 ? -1 : (int32_t)~(uint32_t)k;
                    a.top_logprobs[row * a.top + j - 1] = bad ? nan : k == 0 ? ninf : (value_of(k) - mx) - lse;
                }
                below = k;
            }
        }
    }
}

}  // namespace

cudaError_t launch_logprobs(const DeviceInfo &dev, const LogprobArgs &a, int64_t m, int64_t v, int type,
                            cudaStream_t stream)
{
    return with_type(type, [&](auto t) {
        using T = decltype(t);
        return launch_dependent(logprobs_kernel<T>, dim3((unsigned)(m < (1 << 20) ? m : (1 << 20))), THREADS, 0, stream,
                                a, m, (int)v);
    });
}

}  // namespace q8
