// api.cu -- the extern "C" boundary of libq8act (declared in include/q8act.h): argument
// checks, per-device setup and dispatch to the kernels.  No call allocates memory or
// synchronizes, except q8act_device_status.
#include <mutex>

#include "common.cuh"
#include "launch.h"

namespace {

constexpr int kMaxDevices = 64;

// Device-side status word: kernels OR bits into it when a pipeline wait times out.
__device__ int g_status;

struct DeviceSlot {
    bool ready = false;
    unsigned long long ctx = 0;   // context whose status-word address `info` holds
    int rc = Q8ACT_OK;
    q8::DeviceInfo info{};
};

DeviceSlot g_slots[kMaxDevices];
std::mutex g_mutex;

int cuda_rc(cudaError_t e) { return e == cudaSuccess ? Q8ACT_OK : Q8ACT_ERR_CUDA_BASE + (int)e; }

// Current device's info; checks once per device (and context: the status word's address
// belongs to the context) that it is an sm_103 GPU.
int current_device(const q8::DeviceInfo **out)
{
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_rc(e);
    if (dev < 0 || dev >= kMaxDevices) return Q8ACT_ERR_DEVICE;
    const unsigned long long ctx = q8::current_context_id();
    std::lock_guard<std::mutex> lock(g_mutex);
    DeviceSlot &s = g_slots[dev];
    if (!s.ready || ctx == 0 || ctx != s.ctx) {
        int major = 0, minor = 0, sms = 0, smem = 0;
        if ((e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev)) != cudaSuccess ||
            (e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev)) != cudaSuccess ||
            (e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess ||
            (e = cudaDeviceGetAttribute(&smem, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev)) != cudaSuccess)
            return cuda_rc(e);
        if (major != 10 || minor != 3) {
            s.rc = Q8ACT_ERR_DEVICE;
        } else {
            void *status = nullptr;
            if ((e = cudaGetSymbolAddress(&status, g_status)) != cudaSuccess) return cuda_rc(e);
            s.info.device = dev;
            s.info.num_sms = sms;
            s.info.max_smem_optin = (size_t)smem;
            s.info.status = static_cast<int *>(status);
            s.rc = Q8ACT_OK;
        }
        s.ctx = ctx;
        s.ready = true;
    }
    *out = &s.info;
    return s.rc;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_k(int64_t k)
{
    return (k > 0 && k % q8::K_ALIGN == 0 && k <= Q8ACT_MAX_K) ? Q8ACT_OK : Q8ACT_ERR_DIMS;
}

// Largest m * k the GEMM accepts (keeps every element index inside 32 bits).
constexpr int64_t kMaxGemmElems = (int64_t)1 << 30;

int check_gemm_dims(int64_t m, int64_t n, int64_t k)
{
    if (check_k(k) != Q8ACT_OK || m < 1 || n < 1) return Q8ACT_ERR_DIMS;
    if (m * k > kMaxGemmElems || n * k > ((int64_t)1 << 34) || m * n > ((int64_t)1 << 31))
        return Q8ACT_ERR_DIMS;
    if (n > INT32_MAX || m > INT32_MAX) return Q8ACT_ERR_DIMS;
    return Q8ACT_OK;
}

bool known_type(int type) { return type == Q8ACT_F32 || type == Q8ACT_F16 || type == Q8ACT_BF16; }

int64_t type_size(int type) { return type == Q8ACT_F32 ? 4 : 2; }

// Rows of k elements of a known type, ld elements apart, each 16-byte aligned.
int check_rows(const void *p, int64_t ld, int64_t k, int type)
{
    if (ld < k || ld > ((int64_t)1 << 40)) return Q8ACT_ERR_DIMS;
    return aligned16(p) && ld * type_size(type) % 16 == 0 ? Q8ACT_OK : Q8ACT_ERR_ALIGN;
}

// m x k values of an MXFP4 matrix.
int check_mxfp4_dims(int64_t m, int64_t k)
{
    return check_k(k) == Q8ACT_OK && m >= 1 && m <= INT32_MAX / 2 && m * k <= ((int64_t)1 << 36) ? Q8ACT_OK : Q8ACT_ERR_DIMS;
}

}  // namespace

extern "C" {

int q8act_version(void) { return 100; }

const char *q8act_strerror(int rc)
{
    switch (rc) {
    case Q8ACT_OK: return "ok";
    case Q8ACT_ERR_NULL: return "a required pointer is NULL";
    case Q8ACT_ERR_DIMS: return "dimensions out of range (k must be a positive multiple of 256)";
    case Q8ACT_ERR_ALIGN: return "a pointer is not 16-byte aligned";
    case Q8ACT_ERR_WORKSPACE: return "workspace missing or too small";
    case Q8ACT_ERR_DEVICE: return "the current device is not an sm_103 (GB300) GPU";
    case Q8ACT_ERR_TIMEOUT: return "a kernel timed out waiting in its pipeline";
    case Q8ACT_ERR_TYPE: return "an element type that the call does not take";
    case Q8ACT_ERR_DRAIN_TIMEOUT: return "a kernel timed out waiting for its own copies before exit";
    default:
        if (rc >= Q8ACT_ERR_CUDA_BASE) return cudaGetErrorString((cudaError_t)(rc - Q8ACT_ERR_CUDA_BASE));
        return "unknown error";
    }
}

int64_t q8act_mmq_ldm(int64_t m) { return m < 1 ? 0 : (m + 3) / 4 * 4; }

int q8act_quantize_q8_1(const float *x, int8_t *xq, float *xd, int64_t m, int64_t k, void *stream)
{
    if (!x || !xq || !xd) return Q8ACT_ERR_NULL;
    if (check_k(k) != Q8ACT_OK || m < 1 || m * k > ((int64_t)1 << 34)) return Q8ACT_ERR_DIMS;
    if (!aligned16(x) || !aligned16(xq) || !aligned16(xd)) return Q8ACT_ERR_ALIGN;
    const q8::DeviceInfo *dev;
    int rc = current_device(&dev);
    if (rc) return rc;
    return cuda_rc(q8::launch_quantize_q8_1(*dev, x, xq, xd, m, k, (cudaStream_t)stream));
}

int q8act_quantize_q8_1_mmq(const float *x, uint16_t *xqh, float *xdt, int64_t m, int64_t k, void *stream)
{
    if (!x || !xqh || !xdt) return Q8ACT_ERR_NULL;
    if (check_k(k) != Q8ACT_OK || m < 1 || m * k > kMaxGemmElems) return Q8ACT_ERR_DIMS;
    if (!aligned16(x) || !aligned16(xqh) || !aligned16(xdt)) return Q8ACT_ERR_ALIGN;
    const q8::DeviceInfo *dev;
    int rc = current_device(&dev);
    if (rc) return rc;
    return cuda_rc(q8::launch_quantize_q8_1_mmq(*dev, x, xqh, xdt, m, k, q8act_mmq_ldm(m), (cudaStream_t)stream));
}

int q8act_quantize_q8_0(const float *w, void *wq, int64_t n, int64_t k, void *stream)
{
    if (!w || !wq) return Q8ACT_ERR_NULL;
    if (check_k(k) != Q8ACT_OK || n < 1 || n * k > ((int64_t)1 << 34)) return Q8ACT_ERR_DIMS;
    if (!aligned16(w) || !aligned16(wq)) return Q8ACT_ERR_ALIGN;
    const q8::DeviceInfo *dev;
    int rc = current_device(&dev);
    if (rc) return rc;
    return cuda_rc(q8::launch_quantize_q8_0(*dev, w, static_cast<uint8_t *>(wq), n, k, (cudaStream_t)stream));
}

int q8act_dequant_q8_0_f16(const void *w, void *w16, int64_t n, int64_t k, void *stream)
{
    if (!w || !w16) return Q8ACT_ERR_NULL;
    if (check_k(k) != Q8ACT_OK || n < 1 || n * k > ((int64_t)1 << 34)) return Q8ACT_ERR_DIMS;
    if (!aligned16(w) || !aligned16(w16)) return Q8ACT_ERR_ALIGN;
    const q8::DeviceInfo *dev;
    int rc = current_device(&dev);
    if (rc) return rc;
    return cuda_rc(q8::launch_dequant_q8_0_f16(*dev, static_cast<const uint8_t *>(w), static_cast<uint16_t *>(w16), n, k,
                                               (cudaStream_t)stream));
}

int64_t q8act_repack_ldn(int64_t n) { return n < 1 ? 0 : (n + 3) / 4 * 4; }

int q8act_repack_q8_0(const void *w, uint16_t *wq16, float *wdt, int64_t n, int64_t k, void *stream)
{
    if (!w || !wq16 || !wdt) return Q8ACT_ERR_NULL;
    if (check_k(k) != Q8ACT_OK || n < 1 || n * k > ((int64_t)1 << 34)) return Q8ACT_ERR_DIMS;
    if (!aligned16(w) || !aligned16(wq16) || !aligned16(wdt)) return Q8ACT_ERR_ALIGN;
    const q8::DeviceInfo *dev;
    int rc = current_device(&dev);
    if (rc) return rc;
    return cuda_rc(q8::launch_repack_q8_0(*dev, static_cast<const uint8_t *>(w), wq16, wdt, q8act_repack_ldn(n),
                                          n, k, (cudaStream_t)stream));
}

// pdl: the stream's previous operation is the q8_1 quantizer of the same call; the GEMV is
// then launched as its programmatic dependent.
static int gemv_common(const void *w, const int8_t *xq, const float *xd, float *y, int32_t *dots, int64_t m,
                       int64_t n, int64_t k, void *stream, bool pdl = false)
{
    if (!w || !xq || !xd || (!y && !dots)) return Q8ACT_ERR_NULL;
    if (check_k(k) != Q8ACT_OK || m < 1 || m > Q8ACT_GEMV_MAX_M || n < 1 || n > INT32_MAX / 2 ||
        n * k > ((int64_t)1 << 36))
        return Q8ACT_ERR_DIMS;
    if (!aligned16(w) || !aligned16(xq) || !aligned16(xd) || (y && !aligned16(y)) || (dots && !aligned16(dots)))
        return Q8ACT_ERR_ALIGN;
    const q8::DeviceInfo *dev;
    int rc = current_device(&dev);
    if (rc) return rc;
    if (q8::gemv_mma_supported(*dev, m, k))
        return cuda_rc(q8::launch_gemv_q8_0_mma(*dev, static_cast<const uint8_t *>(w), xq, xd, y, dots, m, n, k,
                                                (cudaStream_t)stream, pdl));
    if (!q8::gemv_supported(*dev, m, k)) return Q8ACT_ERR_DIMS;
    return cuda_rc(q8::launch_gemv_q8_0(*dev, static_cast<const uint8_t *>(w), xq, xd, y, dots, m, n, k,
                                        (cudaStream_t)stream, pdl));
}

int q8act_gemv_q8_0(const void *w, const int8_t *xq, const float *xd, float *y, int64_t m, int64_t n, int64_t k,
                    void *stream)
{
    if (!y) return Q8ACT_ERR_NULL;
    return gemv_common(w, xq, xd, y, nullptr, m, n, k, stream);
}

// Workspace of the fused GEMV: [int8 quants, m * k][f32 scales, m * k / 32], each part
// rounded up to 256 bytes.
size_t q8act_gemv_workspace_bytes(int64_t m, int64_t k)
{
    if (check_k(k) != Q8ACT_OK || m < 1 || m > Q8ACT_GEMV_MAX_M) return 0;
    const size_t quants = (size_t)m * (size_t)k;
    const size_t scales = (size_t)m * (size_t)(k / q8::QK) * 4;
    return ((quants + 255) / 256 * 256) + ((scales + 255) / 256 * 256);
}

int q8act_gemv_q8_0_f32(const void *w, const float *x, float *y, int64_t m, int64_t n, int64_t k, void *ws,
                        size_t ws_bytes, void *stream)
{
    if (!w || !x || !y) return Q8ACT_ERR_NULL;
    if (check_k(k) != Q8ACT_OK || m < 1 || m > Q8ACT_GEMV_MAX_M || n < 1 || n > INT32_MAX / 2 ||
        n * k > ((int64_t)1 << 36))
        return Q8ACT_ERR_DIMS;
    const size_t need = q8act_gemv_workspace_bytes(m, k);
    if (!ws || ws_bytes < need) return Q8ACT_ERR_WORKSPACE;
    if (!aligned16(w) || !aligned16(x) || !aligned16(y) || !aligned16(ws)) return Q8ACT_ERR_ALIGN;
    const q8::DeviceInfo *dev;
    int rc = current_device(&dev);
    if (rc) return rc;
    if (!q8::gemv_mma_supported(*dev, m, k) && !q8::gemv_supported(*dev, m, k)) return Q8ACT_ERR_DIMS;
    int8_t *xq = static_cast<int8_t *>(ws);
    float *xd = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + ((size_t)m * k + 255) / 256 * 256);
    rc = q8act_quantize_q8_1(x, xq, xd, m, k, stream);
    if (rc) return rc;
    return gemv_common(w, xq, xd, y, nullptr, m, n, k, stream, true);
}

int q8act_gemv_q8_0_group(const void *const *w, float *const *y, const int64_t *n, int count, const int8_t *xq,
                          const float *xd, int64_t m, int64_t k, void *stream)
{
    if (!w || !y || !n || !xq || !xd) return Q8ACT_ERR_NULL;
    if (count < 1 || count > Q8ACT_GEMV_MAX_GROUP) return Q8ACT_ERR_DIMS;
    if (check_k(k) != Q8ACT_OK || m < 1 || m > Q8ACT_GEMV_MAX_M) return Q8ACT_ERR_DIMS;
    for (int i = 0; i < count; ++i) {
        if (!w[i] || !y[i]) return Q8ACT_ERR_NULL;
        if (n[i] < 1 || n[i] > INT32_MAX / 2 || n[i] * k > ((int64_t)1 << 36)) return Q8ACT_ERR_DIMS;
        if (!aligned16(w[i]) || !aligned16(y[i])) return Q8ACT_ERR_ALIGN;
    }
    if (!aligned16(xq) || !aligned16(xd)) return Q8ACT_ERR_ALIGN;
    const q8::DeviceInfo *dev;
    int rc = current_device(&dev);
    if (rc) return rc;
    if (q8::gemv_mma_supported(*dev, m, k))
        return cuda_rc(q8::launch_gemv_q8_0_group_mma(*dev, reinterpret_cast<const uint8_t *const *>(w), y, n, count,
                                                      xq, xd, m, k, (cudaStream_t)stream));
    if (!q8::gemv_supported(*dev, m, k)) return Q8ACT_ERR_DIMS;
    return cuda_rc(q8::launch_gemv_q8_0_group(*dev, reinterpret_cast<const uint8_t *const *>(w), y, n, count, xq, xd,
                                              m, k, (cudaStream_t)stream));
}

int q8act_debug_gemv_block_dots(const void *w, const int8_t *xq, int32_t *D, int64_t m, int64_t n, int64_t k,
                                void *stream)
{
    if (!D) return Q8ACT_ERR_NULL;
    // The dot stage needs valid (unused) scales: pass the quants pointer, which is readable.
    return gemv_common(w, xq, reinterpret_cast<const float *>(xq), nullptr, D, m, n, k, stream);
}

// ---- Q4_0 (GGUF 18-byte blocks) ----

int q8act_quantize_q4_0(const float *w, void *wq, int64_t n, int64_t k, void *stream)
{
    if (!w || !wq) return Q8ACT_ERR_NULL;
    if (check_k(k) != Q8ACT_OK || n < 1 || n * k > ((int64_t)1 << 34)) return Q8ACT_ERR_DIMS;
    if (!aligned16(w) || !aligned16(wq)) return Q8ACT_ERR_ALIGN;
    const q8::DeviceInfo *dev;
    int rc = current_device(&dev);
    if (rc) return rc;
    return cuda_rc(q8::launch_quantize_q4_0(*dev, w, static_cast<uint8_t *>(wq), n, k, (cudaStream_t)stream));
}

int q8act_dequant_q4_0_f16(const void *w, void *w16, int64_t n, int64_t k, void *stream)
{
    if (!w || !w16) return Q8ACT_ERR_NULL;
    if (check_k(k) != Q8ACT_OK || n < 1 || n * k > ((int64_t)1 << 34)) return Q8ACT_ERR_DIMS;
    if (!aligned16(w) || !aligned16(w16)) return Q8ACT_ERR_ALIGN;
    const q8::DeviceInfo *dev;
    int rc = current_device(&dev);
    if (rc) return rc;
    return cuda_rc(q8::launch_dequant_q4_0_f16(*dev, static_cast<const uint8_t *>(w), static_cast<uint16_t *>(w16), n, k,
                                               (cudaStream_t)stream));
}

static int gemv_q4_0_common(const void *w, const int8_t *xq, const float *xd, float *y, int32_t *dots, int64_t m,
                            int64_t n, int64_t k, void *stream)
{
    if (!w || !xq || !xd || (!y && !dots)) return Q8ACT_ERR_NULL;
    if (check_k(k) != Q8ACT_OK || m < 1 || m > Q8ACT_GEMV_MAX_M || n < 1 || n > INT32_MAX / 2 ||
        n * k > ((int64_t)1 << 36))
        return Q8ACT_ERR_DIMS;
    if (!aligned16(w) || !aligned16(xq) || !aligned16(xd) || (y && !aligned16(y)) || (dots && !aligned16(dots)))
        return Q8ACT_ERR_ALIGN;
    const q8::DeviceInfo *dev;
    int rc = current_device(&dev);
    if (rc) return rc;
    if (q8::gemv_q4_0_mma_supported(*dev, m, k))
        return cuda_rc(q8::launch_gemv_q4_0_mma(*dev, static_cast<const uint8_t *>(w), xq, xd, y, dots, m, n, k,
                                                (cudaStream_t)stream));
    if (!q8::gemv_q4_0_supported(*dev, m, k)) return Q8ACT_ERR_DIMS;
    return cuda_rc(q8::launch_gemv_q4_0(*dev, static_cast<const uint8_t *>(w), xq, xd, y, dots, m, n, k,
                                        (cudaStream_t)stream));
}

int q8act_gemv_q4_0(const void *w, const int8_t *xq, const float *xd, float *y, int64_t m, int64_t n, int64_t k,
                    void *stream)
{
    if (!y) return Q8ACT_ERR_NULL;
    return gemv_q4_0_common(w, xq, xd, y, nullptr, m, n, k, stream);
}

int q8act_debug_gemv_q4_0_block_dots(const void *w, const int8_t *xq, int32_t *D, int64_t m, int64_t n, int64_t k,
                                     void *stream)
{
    if (!D) return Q8ACT_ERR_NULL;
    // As for Q8_0: the dot stage reads (and ignores) a scale array; the quants are readable.
    return gemv_q4_0_common(w, xq, reinterpret_cast<const float *>(xq), nullptr, D, m, n, k, stream);
}

// ---- K-quant superblocks (GGUF Q6_K 210 B, Q4_K 144 B, Q5_K 176 B; 256 weights each) ----

static int dequant_kq_common(int fmt, const void *w, void *w16, int64_t n, int64_t k, void *stream)
{
    if (!w || !w16) return Q8ACT_ERR_NULL;
    if (check_k(k) != Q8ACT_OK || n < 1 || n > INT32_MAX || n * k > ((int64_t)1 << 34)) return Q8ACT_ERR_DIMS;
    if (!aligned16(w) || !aligned16(w16)) return Q8ACT_ERR_ALIGN;
    const q8::DeviceInfo *dev;
    int rc = current_device(&dev);
    if (rc) return rc;
    return cuda_rc(q8::launch_dequant_kq_f16(*dev, fmt, static_cast<const uint8_t *>(w), static_cast<uint16_t *>(w16),
                                             n, k, (cudaStream_t)stream));
}

int q8act_dequant_q6_k_f16(const void *w, void *w16, int64_t n, int64_t k, void *stream)
{
    return dequant_kq_common(6, w, w16, n, k, stream);
}
int q8act_dequant_q4_k_f16(const void *w, void *w16, int64_t n, int64_t k, void *stream)
{
    return dequant_kq_common(4, w, w16, n, k, stream);
}
int q8act_dequant_q5_k_f16(const void *w, void *w16, int64_t n, int64_t k, void *stream)
{
    return dequant_kq_common(5, w, w16, n, k, stream);
}

static int gemv_kq_common(int fmt, const void *w, const int8_t *xq, const float *xd, float *y, int32_t *dots,
                          int64_t m, int64_t n, int64_t k, void *stream)
{
    if (!w || !xq || !xd || (!y && !dots)) return Q8ACT_ERR_NULL;
    if (check_k(k) != Q8ACT_OK || m < 1 || m > Q8ACT_GEMV_KQ_MAX_M || n < 1 || n > INT32_MAX / 2 ||
        n * k > ((int64_t)1 << 36))
        return Q8ACT_ERR_DIMS;
    if (!aligned16(w) || !aligned16(xq) || !aligned16(xd) || (y && !aligned16(y)) || (dots && !aligned16(dots)))
        return Q8ACT_ERR_ALIGN;
    const q8::DeviceInfo *dev;
    int rc = current_device(&dev);
    if (rc) return rc;
    if (!q8::gemv_kq_supported(*dev, fmt, m, k)) return Q8ACT_ERR_DIMS;
    return cuda_rc(q8::launch_gemv_kq(*dev, fmt, static_cast<const uint8_t *>(w), xq, xd, y, dots, m, n, k,
                                      (cudaStream_t)stream));
}

int q8act_gemv_q6_k(const void *w, const int8_t *xq, const float *xd, float *y, int64_t m, int64_t n, int64_t k,
                    void *stream)
{
    if (!y) return Q8ACT_ERR_NULL;
    return gemv_kq_common(6, w, xq, xd, y, nullptr, m, n, k, stream);
}
int q8act_gemv_q4_k(const void *w, const int8_t *xq, const float *xd, float *y, int64_t m, int64_t n, int64_t k,
                    void *stream)
{
    if (!y) return Q8ACT_ERR_NULL;
    return gemv_kq_common(4, w, xq, xd, y, nullptr, m, n, k, stream);
}
int q8act_gemv_q5_k(const void *w, const int8_t *xq, const float *xd, float *y, int64_t m, int64_t n, int64_t k,
                    void *stream)
{
    if (!y) return Q8ACT_ERR_NULL;
    return gemv_kq_common(5, w, xq, xd, y, nullptr, m, n, k, stream);
}

// The block-integer stage needs a readable scale array; the quants are readable and larger.
int q8act_debug_gemv_q6_k_block_dots(const void *w, const int8_t *xq, int32_t *D, int64_t m, int64_t n, int64_t k,
                                     void *stream)
{
    if (!D) return Q8ACT_ERR_NULL;
    return gemv_kq_common(6, w, xq, reinterpret_cast<const float *>(xq), nullptr, D, m, n, k, stream);
}
int q8act_debug_gemv_q4_k_block_dots(const void *w, const int8_t *xq, int32_t *D, int64_t m, int64_t n, int64_t k,
                                     void *stream)
{
    if (!D) return Q8ACT_ERR_NULL;
    return gemv_kq_common(4, w, xq, reinterpret_cast<const float *>(xq), nullptr, D, m, n, k, stream);
}
int q8act_debug_gemv_q5_k_block_dots(const void *w, const int8_t *xq, int32_t *D, int64_t m, int64_t n, int64_t k,
                                     void *stream)
{
    if (!D) return Q8ACT_ERR_NULL;
    return gemv_kq_common(5, w, xq, reinterpret_cast<const float *>(xq), nullptr, D, m, n, k, stream);
}

// Workspace of the fused GEMMs: [binary16 quants][block-major scales][split region].  The
// first two are required; with the split region as well, a launch may take the balanced
// schedule (equal runs of (tile, k group) units per CTA, tiles cut into k pieces at the runs'
// ends).
static size_t act_bytes(int64_t m, int64_t k)
{
    const size_t quants = (size_t)m * (size_t)k * 2;
    const size_t scales = (size_t)(k / q8::QK) * (size_t)q8act_mmq_ldm(m) * 4;
    return ((quants + 255) / 256 * 256) + ((scales + 255) / 256 * 256);
}

size_t q8act_gemm_workspace_bytes(int64_t m, int64_t k)
{
    if (check_k(k) != Q8ACT_OK || m < 1 || m * k > kMaxGemmElems) return 0;
    return act_bytes(m, k) + Q8ACT_GEMM_SPLIT_BYTES;
}

// pdl: the stream's previous operation is the MMQ quantizer of the same call, enqueued after
// q8::gemm_prepare_split; the GEMM is then launched as its programmatic dependent.
static int gemm_core(const void *w, const uint16_t *xqh, const float *xdt, float *y, int32_t *dots, int64_t m,
                     int64_t n, int64_t k, void *split_ws, size_t split_bytes, bool pdl, void *stream)
{
    if (!w || !xqh || !xdt || (!y && !dots)) return Q8ACT_ERR_NULL;
    if (check_gemm_dims(m, n, k) != Q8ACT_OK) return Q8ACT_ERR_DIMS;
    if (!aligned16(w) || !aligned16(xqh) || !aligned16(xdt) || (y && !aligned16(y)) || (dots && !aligned16(dots)))
        return Q8ACT_ERR_ALIGN;
    const q8::DeviceInfo *dev;
    int rc = current_device(&dev);
    if (rc) return rc;
    return cuda_rc(q8::launch_gemm_q8_0(*dev, static_cast<const uint8_t *>(w), xqh, xdt, y, dots, m, n, k,
                                        q8act_mmq_ldm(m), split_ws, split_bytes, pdl, (cudaStream_t)stream));
}

int q8act_gemm_q8_0(const void *w, const float *x, float *y, int64_t m, int64_t n, int64_t k, void *ws,
                    size_t ws_bytes, void *stream)
{
    if (!w || !x || !y) return Q8ACT_ERR_NULL;
    if (check_gemm_dims(m, n, k) != Q8ACT_OK) return Q8ACT_ERR_DIMS;
    const size_t need = act_bytes(m, k);
    if (!ws || ws_bytes < need) return Q8ACT_ERR_WORKSPACE;
    if (!aligned16(w) || !aligned16(x) || !aligned16(y) || !aligned16(ws)) return Q8ACT_ERR_ALIGN;
    uint16_t *xqh = static_cast<uint16_t *>(ws);
    float *xdt = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + ((size_t)m * k * 2 + 255) / 256 * 256);
    void *split_ws = static_cast<uint8_t *>(ws) + need;
    const q8::DeviceInfo *dev;
    int rc = current_device(&dev);
    if (rc) return rc;
    rc = cuda_rc(q8::gemm_prepare_split(*dev, m, n, k, false, split_ws, ws_bytes - need, (cudaStream_t)stream));
    if (rc) return rc;
    rc = q8act_quantize_q8_1_mmq(x, xqh, xdt, m, k, stream);
    if (rc) return rc;
    return gemm_core(w, xqh, xdt, y, nullptr, m, n, k, split_ws, ws_bytes - need, true, stream);
}

int q8act_gemm_q8_0_preq(const void *w, const uint16_t *xqh, const float *xdt, float *y, int64_t m, int64_t n,
                         int64_t k, void *stream)
{
    if (!y) return Q8ACT_ERR_NULL;
    return gemm_core(w, xqh, xdt, y, nullptr, m, n, k, nullptr, 0, false, stream);
}

static int gemm_repacked_core(const uint16_t *wq16, const float *wdt, const uint16_t *xqh, const float *xdt,
                              float *y, int32_t *dots, int64_t m, int64_t n, int64_t k, void *split_ws,
                              size_t split_bytes, bool pdl, void *stream)
{
    if (!wq16 || !wdt || !xqh || !xdt || (!y && !dots)) return Q8ACT_ERR_NULL;
    if (check_gemm_dims(m, n, k) != Q8ACT_OK) return Q8ACT_ERR_DIMS;
    if (!aligned16(wq16) || !aligned16(wdt) || !aligned16(xqh) || !aligned16(xdt) || (y && !aligned16(y)) ||
        (dots && !aligned16(dots)))
        return Q8ACT_ERR_ALIGN;
    const q8::DeviceInfo *dev;
    int rc = current_device(&dev);
    if (rc) return rc;
    return cuda_rc(q8::launch_gemm_q8_0_repacked(*dev, wq16, wdt, q8act_repack_ldn(n), xqh, xdt, y, dots, m, n, k,
                                                 q8act_mmq_ldm(m), split_ws, split_bytes, pdl, (cudaStream_t)stream));
}

int q8act_gemm_q8_0_repacked(const uint16_t *wq16, const float *wdt, const float *x, float *y, int64_t m,
                             int64_t n, int64_t k, void *ws, size_t ws_bytes, void *stream)
{
    if (!wq16 || !wdt || !x || !y) return Q8ACT_ERR_NULL;
    if (check_gemm_dims(m, n, k) != Q8ACT_OK) return Q8ACT_ERR_DIMS;
    const size_t need = act_bytes(m, k);
    if (!ws || ws_bytes < need) return Q8ACT_ERR_WORKSPACE;
    if (!aligned16(wq16) || !aligned16(wdt) || !aligned16(x) || !aligned16(y) || !aligned16(ws))
        return Q8ACT_ERR_ALIGN;
    uint16_t *xqh = static_cast<uint16_t *>(ws);
    float *xdt = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + ((size_t)m * k * 2 + 255) / 256 * 256);
    void *split_ws = static_cast<uint8_t *>(ws) + need;
    const q8::DeviceInfo *dev;
    int rc = current_device(&dev);
    if (rc) return rc;
    rc = cuda_rc(q8::gemm_prepare_split(*dev, m, n, k, true, split_ws, ws_bytes - need, (cudaStream_t)stream));
    if (rc) return rc;
    rc = q8act_quantize_q8_1_mmq(x, xqh, xdt, m, k, stream);
    if (rc) return rc;
    return gemm_repacked_core(wq16, wdt, xqh, xdt, y, nullptr, m, n, k, split_ws, ws_bytes - need, true, stream);
}

int q8act_debug_gemm_repacked_block_dots(const uint16_t *wq16, const float *wdt, const uint16_t *xqh, int32_t *D,
                                         int64_t m, int64_t n, int64_t k, void *stream)
{
    if (!D) return Q8ACT_ERR_NULL;
    // The dot stage needs a readable (unused) activation-scale array: reuse the quants.
    return gemm_repacked_core(wq16, wdt, xqh, reinterpret_cast<const float *>(xqh), nullptr, D, m, n, k, nullptr, 0,
                              false, stream);
}

int q8act_debug_gemm_block_dots(const void *w, const uint16_t *xqh, int32_t *D, int64_t m, int64_t n, int64_t k,
                                void *stream)
{
    if (!D) return Q8ACT_ERR_NULL;
    // The dot stage needs a readable (unused) scale array of the right shape: reuse the
    // quants, which are larger than the scale array.
    return gemm_core(w, xqh, reinterpret_cast<const float *>(xqh), nullptr, D, m, n, k, nullptr, 0, false, stream);
}

// ---- the norm in front of a product ----

static int rmsnorm_common(const void *x, int64_t ldx, const void *residual, int64_t ldr, const void *weight, int wtype,
                          float eps, void *residual_out, int64_t ldro, void *y, void *q, float *d, bool mmq, int64_t m,
                          int64_t k, int type, void *stream)
{
    if (!x || !q != !d || (!q && !y)) return Q8ACT_ERR_NULL;
    if (!known_type(type) || (weight && !known_type(wtype))) return Q8ACT_ERR_TYPE;
    if (check_k(k) != Q8ACT_OK || m < 1 || m > ((int64_t)1 << 34) / k || !(eps >= 0.0f)) return Q8ACT_ERR_DIMS;
    if (mmq && m * k > kMaxGemmElems) return Q8ACT_ERR_DIMS;
    int rc = check_rows(x, ldx, k, type);
    if (!rc && residual) rc = check_rows(residual, ldr, k, type);
    if (!rc && residual_out) rc = check_rows(residual_out, ldro, k, type);
    if (rc) return rc;
    if (!aligned16(weight) || !aligned16(y) || !aligned16(q) || !aligned16(d)) return Q8ACT_ERR_ALIGN;
    const q8::DeviceInfo *dev;
    if ((rc = current_device(&dev))) return rc;
    const q8::NormArgs a{x, residual, weight, residual_out, y, q, d, ldx, ldr, ldro, q8act_mmq_ldm(m), eps, 1.0f / (float)k, wtype};
    return cuda_rc(q8::launch_rmsnorm_q8_1(*dev, a, mmq, m, k, type, (cudaStream_t)stream));
}

int q8act_rmsnorm_q8_1(const void *x, int64_t ldx, const void *residual, int64_t ldr, const void *weight, int wtype,
                       float eps, void *residual_out, int64_t ldro, void *y, int8_t *xq, float *xd, int64_t m,
                       int64_t k, int type, void *stream)
{
    return rmsnorm_common(x, ldx, residual, ldr, weight, wtype, eps, residual_out, ldro, y, xq, xd, false, m, k, type,
                          stream);
}

int q8act_rmsnorm_q8_1_mmq(const void *x, int64_t ldx, const void *residual, int64_t ldr, const void *weight,
                           int wtype, float eps, void *residual_out, int64_t ldro, void *y, uint16_t *xqh, float *xdt,
                           int64_t m, int64_t k, int type, void *stream)
{
    return rmsnorm_common(x, ldx, residual, ldr, weight, wtype, eps, residual_out, ldro, y, xqh, xdt, true, m, k, type,
                          stream);
}

// ---- MXFP4 ----

size_t q8act_mxfp4_scale_bytes(int64_t rows, int64_t k)
{
    if (check_mxfp4_dims(rows, k) != Q8ACT_OK) return 0;
    return (size_t)((rows + 127) / 128) * (size_t)(k / 128) * 512;
}

int q8act_quantize_mxfp4(const void *x, int64_t ldx, int type, void *codes, void *scales, int64_t m, int64_t k,
                         void *stream)
{
    if (!x || !codes || !scales) return Q8ACT_ERR_NULL;
    if (!known_type(type)) return Q8ACT_ERR_TYPE;
    if (check_mxfp4_dims(m, k) != Q8ACT_OK) return Q8ACT_ERR_DIMS;
    int rc = check_rows(x, ldx, k, type);
    if (rc) return rc;
    if (!aligned16(codes) || !aligned16(scales)) return Q8ACT_ERR_ALIGN;
    const q8::DeviceInfo *dev;
    if ((rc = current_device(&dev))) return rc;
    return cuda_rc(q8::launch_quantize_mxfp4(*dev, x, ldx, type, static_cast<uint8_t *>(codes),
                                             static_cast<uint8_t *>(scales), m, k, (cudaStream_t)stream));
}

int q8act_dequant_mxfp4(const void *codes, const void *scales, void *y, int type, int64_t m, int64_t k, void *stream)
{
    if (!codes || !scales || !y) return Q8ACT_ERR_NULL;
    if (!known_type(type)) return Q8ACT_ERR_TYPE;
    if (check_mxfp4_dims(m, k) != Q8ACT_OK) return Q8ACT_ERR_DIMS;
    if (!aligned16(codes) || !aligned16(scales) || !aligned16(y)) return Q8ACT_ERR_ALIGN;
    const q8::DeviceInfo *dev;
    int rc = current_device(&dev);
    if (rc) return rc;
    return cuda_rc(q8::launch_dequant_mxfp4(*dev, static_cast<const uint8_t *>(codes),
                                            static_cast<const uint8_t *>(scales), y, type, m, k, (cudaStream_t)stream));
}

int q8act_tile_mxfp4_scales(const void *scales, void *tiled, int64_t m, int64_t k, void *stream)
{
    if (!scales || !tiled) return Q8ACT_ERR_NULL;
    if (check_mxfp4_dims(m, k) != Q8ACT_OK) return Q8ACT_ERR_DIMS;
    if (!aligned16(scales) || !aligned16(tiled)) return Q8ACT_ERR_ALIGN;
    const q8::DeviceInfo *dev;
    int rc = current_device(&dev);
    if (rc) return rc;
    return cuda_rc(q8::launch_tile_mxfp4_scales(*dev, static_cast<const uint8_t *>(scales),
                                                static_cast<uint8_t *>(tiled), m, k, (cudaStream_t)stream));
}

// Workspace of the fused product: the activation's codes, rounded up to 256 bytes, then its scales.
size_t q8act_gemm_mxfp4_workspace_bytes(int64_t m, int64_t k)
{
    if (check_mxfp4_dims(m, k) != Q8ACT_OK) return 0;
    return ((size_t)m * k / 2 + 255) / 256 * 256 + q8act_mxfp4_scale_bytes(m, k);
}

static int gemm_mxfp4_check(int ytype, int64_t m, int64_t n, int64_t k)
{
    if (!known_type(ytype)) return Q8ACT_ERR_TYPE;
    if (check_mxfp4_dims(m, k) != Q8ACT_OK || check_mxfp4_dims(n, k) != Q8ACT_OK) return Q8ACT_ERR_DIMS;
    return m * n <= ((int64_t)1 << 40) ? Q8ACT_OK : Q8ACT_ERR_DIMS;
}

// pdl: the stream's previous operation is the quantizer of the same call.
static int gemm_mxfp4_core(const void *w, const void *wscales, const void *xq, const void *xscales, void *y, int ytype,
                           int64_t m, int64_t n, int64_t k, bool pdl, void *stream)
{
    if (!w || !wscales || !xq || !xscales || !y) return Q8ACT_ERR_NULL;
    int rc = gemm_mxfp4_check(ytype, m, n, k);
    if (rc) return rc;
    if (!aligned16(w) || !aligned16(wscales) || !aligned16(xq) || !aligned16(xscales) || !aligned16(y))
        return Q8ACT_ERR_ALIGN;
    const q8::DeviceInfo *dev;
    if ((rc = current_device(&dev))) return rc;
    return cuda_rc(q8::launch_gemm_mxfp4(*dev, static_cast<const uint8_t *>(w), static_cast<const uint8_t *>(wscales),
                                         static_cast<const uint8_t *>(xq), static_cast<const uint8_t *>(xscales), y,
                                         ytype, m, n, k, pdl, (cudaStream_t)stream));
}

int q8act_gemm_mxfp4_preq(const void *w, const void *wscales, const void *xq, const void *xscales, void *y, int ytype,
                          int64_t m, int64_t n, int64_t k, void *stream)
{
    return gemm_mxfp4_core(w, wscales, xq, xscales, y, ytype, m, n, k, false, stream);
}

int q8act_gemm_mxfp4(const void *w, const void *wscales, const void *x, int64_t ldx, int xtype, void *y, int ytype,
                     int64_t m, int64_t n, int64_t k, void *ws, size_t ws_bytes, void *stream)
{
    if (!w || !wscales || !x || !y) return Q8ACT_ERR_NULL;
    if (!known_type(xtype)) return Q8ACT_ERR_TYPE;
    int rc = gemm_mxfp4_check(ytype, m, n, k);
    if (rc) return rc;
    if (!ws || ws_bytes < q8act_gemm_mxfp4_workspace_bytes(m, k)) return Q8ACT_ERR_WORKSPACE;
    if (!aligned16(w) || !aligned16(wscales) || !aligned16(y) || !aligned16(ws)) return Q8ACT_ERR_ALIGN;
    if ((rc = check_rows(x, ldx, k, xtype))) return rc;
    const q8::DeviceInfo *dev;
    if ((rc = current_device(&dev))) return rc;
    if (q8::gemm_mxfp4_quantizes(dev->num_sms, m, n, k))
        return cuda_rc(q8::launch_gemm_mxfp4_own(*dev, static_cast<const uint8_t *>(w),
                                                 static_cast<const uint8_t *>(wscales), x, ldx, xtype, y, ytype, m, n, k,
                                                 (cudaStream_t)stream));
    uint8_t *xq = static_cast<uint8_t *>(ws), *xsc = xq + ((size_t)m * k / 2 + 255) / 256 * 256;
    rc = q8act_quantize_mxfp4(x, ldx, xtype, xq, xsc, m, k, stream);
    if (rc) return rc;
    return gemm_mxfp4_core(w, wscales, xq, xsc, y, ytype, m, n, k, true, stream);
}

// Test hook, host only: the choice that the MXFP4 products make.
int q8act_debug_gemm_mxfp4_plan(int sms, int64_t m, int64_t n, int64_t k, int32_t *plan)
{
    if (!plan) return Q8ACT_ERR_NULL;
    const int rc = gemm_mxfp4_check(Q8ACT_F32, m, n, k);
    if (rc) return rc;
    if (sms < 32 || sms > 1024) return Q8ACT_ERR_DIMS;
    const q8::GemmPlan p = q8::gemm_mxfp4_plan(sms, m, n, k);
    plan[0] = p.bn;
    plan[1] = p.CL;
    plan[2] = p.per_sm;
    plan[3] = q8::gemm_mxfp4_quantizes(sms, m, n, k);
    return Q8ACT_OK;
}

// ---- log probabilities ----

int q8act_logprobs(const void *logits, int64_t ld, int type, const int32_t *tokens, float *logprob, float *entropy,
                   int32_t *top_ids, float *top_logprobs, int64_t m, int64_t v, int top, void *stream)
{
    if (!logits || !tokens != !logprob || (top > 0 && (!top_ids || !top_logprobs))) return Q8ACT_ERR_NULL;
    if (!known_type(type)) return Q8ACT_ERR_TYPE;
    if (m < 1 || v < 1 || v > (1 << 30) || top < 0 || top > Q8ACT_MAX_TOP || ld < v || ld > ((int64_t)1 << 40) ||
        m > ((int64_t)1 << 46) / ld)
        return Q8ACT_ERR_DIMS;
    // Rows start wherever ld puts them, so the arrays need their elements' alignment only.
    const uintptr_t words = (uintptr_t)tokens | (uintptr_t)logprob | (uintptr_t)entropy | (uintptr_t)top_ids |
                            (uintptr_t)top_logprobs;
    if ((uintptr_t)logits % type_size(type) || words % 4) return Q8ACT_ERR_ALIGN;
    const q8::DeviceInfo *dev;
    int rc = current_device(&dev);
    if (rc) return rc;
    const q8::LogprobArgs a{logits, tokens, logprob, entropy, top_ids, top_logprobs, ld, top};
    return cuda_rc(q8::launch_logprobs(*dev, a, m, v, type, (cudaStream_t)stream));
}

// ---- the paged key/value cache ----

static bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// The batch, for m rows of heads_q query heads.
static int check_paged(const q8act_paged_kv *kv, int64_t m, int64_t heads_q)
{
    if (!kv || !kv->k || !kv->v || !kv->table || !kv->starts || !kv->lens) return Q8ACT_ERR_NULL;
    if (kv->type != Q8ACT_F16 && kv->type != Q8ACT_BF16) return Q8ACT_ERR_TYPE;
    const int64_t ps = kv->page_size;
    if ((kv->dim != 64 && kv->dim != 128) || ps < 16 || ps > 1024 || (ps & (ps - 1)) || kv->heads < 1 || kv->heads > 1024 ||
        kv->pages < 1 || kv->pages >= INT32_MAX || kv->page_stride < kv->heads * ps * kv->dim ||
        kv->page_stride >= ((int64_t)1 << 38) || kv->seqs < 1 || kv->seqs > (1 << 16) || kv->table_width < 1 ||
        kv->table_width * ps > (1 << 30) || kv->table_ld < kv->table_width || kv->table_ld >= ((int64_t)1 << 40))
        return Q8ACT_ERR_DIMS;
    if (m < 1 || heads_q < 0 || heads_q > 4096 || m * (heads_q + 2 * kv->heads) > (1 << 30)) return Q8ACT_ERR_DIMS;
    if (!aligned16(kv->k) || !aligned16(kv->v) || kv->page_stride % 8 || !aligned4(kv->table) || !aligned4(kv->starts) ||
        !aligned4(kv->lens))
        return Q8ACT_ERR_ALIGN;
    return Q8ACT_OK;
}

// m rows of token values in memory, in bytes.
struct Rows {
    intptr_t at;
    int64_t ld, size;
};
static Rows rows_of(const void *p, int64_t ld, int64_t values, int type)
{
    return Rows{reinterpret_cast<intptr_t>(p), ld * type_size(type), values * type_size(type)};
}

// Whether m rows of a and of b share a byte (rows equally far apart: exactly; otherwise where one begins before the other's end).
// Beside each other in the same wider rows they do not.
static bool rows_overlap(const Rows &a, const Rows &b, int64_t m)
{
    using Wide = __int128;                       // m and distances of 2^40 elements pass 64 bits
    auto end = [&](const Rows &r) { return (Wide)r.at + (Wide)(m - 1) * r.ld + r.size; };
    if (a.at >= end(b) || b.at >= end(a)) return false;
    if (m == 1 || a.ld != b.ld) return true;
    const Wide d = (((Wide)b.at - a.at) % a.ld + a.ld) % a.ld;       // from a row of a to the next beginning of one of b
    return d < a.size || d + b.size > a.ld;
}

int q8act_append_kv(const q8act_paged_kv *kv, const void *q, int64_t ldq, const void *k, int64_t ldk, const void *v,
                    int64_t ldv, int type, void *q_out, int64_t ldqo, int heads_q, const uint64_t *turns, int rot,
                    int interleaved, int64_t m, void *stream)
{
    if (!k || !v || !q != !q_out || !q != !heads_q || !turns != !rot) return Q8ACT_ERR_NULL;
    if (m < 1 || m > (1 << 30)) return Q8ACT_ERR_DIMS;
    int rc = check_paged(kv, m, heads_q);
    if (rc) return rc;
    if (!known_type(type)) return Q8ACT_ERR_TYPE;
    if (rot < 0 || rot > kv->dim || rot % 16 || (interleaved != 0 && interleaved != 1)) return Q8ACT_ERR_DIMS;
    if ((rc = check_rows(k, ldk, (int64_t)kv->heads * kv->dim, type)) ||
        (rc = check_rows(v, ldv, (int64_t)kv->heads * kv->dim, type)))
        return rc;
    if (q && ((rc = check_rows(q, ldq, (int64_t)heads_q * kv->dim, type)) ||
              (rc = check_rows(q_out, ldqo, (int64_t)heads_q * kv->dim, kv->type))))
        return rc;
    if (q && q == q_out && type != kv->type) return Q8ACT_ERR_TYPE;
    if (q && q == q_out && ldq != ldqo) return Q8ACT_ERR_DIMS;
    if (q) {             // a thread writes the 16 values that it has read, and no others
        const int64_t n = (int64_t)kv->heads * kv->dim, nq = (int64_t)heads_q * kv->dim;
        const Rows o = rows_of(q_out, ldqo, nq, kv->type);
        if ((q != q_out && rows_overlap(rows_of(q, ldq, nq, type), o, m)) || rows_overlap(rows_of(k, ldk, n, type), o, m) ||
            rows_overlap(rows_of(v, ldv, n, type), o, m))
            return Q8ACT_ERR_DIMS;
    }
    if (reinterpret_cast<uintptr_t>(turns) & 7u) return Q8ACT_ERR_ALIGN;
    const q8::DeviceInfo *dev;
    if ((rc = current_device(&dev))) return rc;
    const q8::AppendArgs a{q, k, v, q_out, ldq, ldk, ldv, ldqo, turns, type, heads_q, rot, interleaved};
    return cuda_rc(q8::launch_append_kv(*dev, *kv, a, m, (cudaStream_t)stream));
}

static bool attention_heads(int64_t heads_q, int64_t heads, int64_t dim)
{
    return heads >= 1 && heads <= 1024 && heads_q >= heads && heads_q <= 4096 && heads_q % heads == 0 &&
           (dim == 64 || dim == 128);
}

size_t q8act_attention_workspace_bytes(int heads_q, int heads, int dim)
{
    return attention_heads(heads_q, heads, dim) ? q8::attention_workspace_bytes(dim) : 0;
}

int q8act_attention(const q8act_paged_kv *kv, const void *q, int64_t ldq, void *out, int64_t ldo, int otype, int heads_q,
                    float scale, int window, int max_new, int64_t m, void *ws, size_t ws_bytes, void *stream)
{
    if (!q || !out) return Q8ACT_ERR_NULL;
    if (m < 1 || m > (1 << 30)) return Q8ACT_ERR_DIMS;
    int rc = check_paged(kv, m, heads_q);
    if (rc) return rc;
    if (!known_type(otype)) return Q8ACT_ERR_TYPE;
    if (!attention_heads(heads_q, kv->heads, kv->dim) || !(scale > 0.0f) || scale > 0x1p100f || window < 0 ||
        window > (1 << 30) || max_new < 0)
        return Q8ACT_ERR_DIMS;
    if ((rc = check_rows(q, ldq, (int64_t)heads_q * kv->dim, kv->type)) ||
        (rc = check_rows(out, ldo, (int64_t)heads_q * kv->dim, otype)))
        return rc;
    // (a unit's output may be written before another one has read its queries)
    if (rows_overlap(rows_of(q, ldq, (int64_t)heads_q * kv->dim, kv->type), rows_of(out, ldo, (int64_t)heads_q * kv->dim, otype), m))
        return Q8ACT_ERR_DIMS;
    if (!ws || ws_bytes < q8::attention_workspace_bytes(kv->dim)) return Q8ACT_ERR_WORKSPACE;
    if (!aligned16(ws)) return Q8ACT_ERR_ALIGN;
    const q8::DeviceInfo *dev;
    if ((rc = current_device(&dev))) return rc;
    const q8::AttentionArgs a{q, out, ws, ldq, ldo, otype, heads_q, window, max_new, scale};
    return cuda_rc(q8::launch_attention(*dev, *kv, a, m, (cudaStream_t)stream));
}

// Test hook: one thread waits on an mbarrier that nothing arrives on, through the pipelines'
// own bounded wait, until limit_ns passes; the wait then records STATUS_TIMEOUT.  Nothing
// else is in flight (no copies, no tensor-core work), so the exit is clean.
__global__ void wait_timeout_kernel(unsigned long long limit_ns, int *status)
{
    __shared__ uint64_t bar;
    if (threadIdx.x == 0) {
        q8::mbar_init(&bar, 1);
        q8::fence_mbar_init();
        q8::mbar_wait_for(&bar, 0, status, limit_ns, q8::STATUS_TIMEOUT);
        asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(q8::smem_u32(&bar)) : "memory");
    }
}

int q8act_debug_wait_timeout(int64_t limit_ns, void *stream)
{
    if (limit_ns < 1000 || limit_ns > 1000000000) return Q8ACT_ERR_DIMS;
    const q8::DeviceInfo *dev;
    int rc = current_device(&dev);
    if (rc) return rc;
    wait_timeout_kernel<<<1, 32, 0, (cudaStream_t)stream>>>((unsigned long long)limit_ns, dev->status);
    return cuda_rc(cudaGetLastError());
}

int q8act_device_status(void *stream)
{
    const q8::DeviceInfo *dev;
    int rc = current_device(&dev);
    if (rc) return rc;
    cudaError_t e = cudaStreamSynchronize((cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_rc(e);
    int host = 0;
    const int zero = 0;
    if ((e = cudaMemcpyFromSymbol(&host, g_status, sizeof(int))) != cudaSuccess) return cuda_rc(e);
    if (host && (e = cudaMemcpyToSymbol(g_status, &zero, sizeof(int))) != cudaSuccess) return cuda_rc(e);
    if (host & q8::STATUS_DRAIN_TIMEOUT) return Q8ACT_ERR_DRAIN_TIMEOUT;
    return host ? Q8ACT_ERR_TIMEOUT : Q8ACT_OK;
}

}  // extern "C"
