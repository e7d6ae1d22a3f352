// abi.hip -- the C ABI of libbitnet_i2s.so (declared in include/bitnet_i2s.h):
// host-side argument validation, error reporting and kernel dispatch.
#include <stdarg.h>
#include <stdio.h>

#include <algorithm>
#include <initializer_list>
#include <mutex>
#include <string>

#include "bitnet_i2s.h"
#include "common.h"
#include "layer.h"

#define BITNET_API extern "C" __attribute__((visibility("default")))

#ifndef BITNET_VALU_MAX_N
#define BITNET_VALU_MAX_N 2   // decode token counts served by the vector-ALU GEMV (MFMA above)
#endif

namespace {

thread_local std::string g_last_error;

int fail(int status, const char *fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    g_last_error = buf;
    return status;
}

int ok() {
    g_last_error.clear();
    return BITNET_OK;
}

int hip_fail(const char *where, hipError_t e) {
    return fail(BITNET_E_HIP, "%s: %s (%d)", where, hipGetErrorString(e), (int)e);
}

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

int check_k(const char *fn, int64_t K) {
    if (K <= 0 || K % bitnet::kBlock != 0 || K > BITNET_MAX_K)
        return fail(BITNET_E_SHAPE, "%s: K=%lld must be a positive multiple of 128 and <= %d",
                    fn, (long long)K, BITNET_MAX_K);
    return BITNET_OK;
}

// Device-side count of non-ternary weights seen by the packer.  Each device
// holds its own copy; its address is looked up once per device with
// hipGetSymbolAddress and only that address is used from the host.
__device__ unsigned g_pack_bad;
constexpr int kMaxDevices = 64;
void *g_pack_bad_addr[kMaxDevices];
std::mutex g_pack_mu;

int pack_counter(int dev, unsigned **out) {
    if (dev < 0 || dev >= kMaxDevices)
        return fail(BITNET_E_HIP, "bitnet_pack_i2s: device index %d unsupported", dev);
    if (!g_pack_bad_addr[dev]) {
        void *p = nullptr;
        hipError_t e = hipGetSymbolAddress(&p, HIP_SYMBOL(g_pack_bad));
        if (e != hipSuccess) return hip_fail("bitnet_pack_i2s: hipGetSymbolAddress", e);
        g_pack_bad_addr[dev] = p;
    }
    *out = static_cast<unsigned *>(g_pack_bad_addr[dev]);
    return BITNET_OK;
}

// Scratch of the one-time weight conversion calls (AbsMean partial sums, the
// scale, the non-finite count and max|w|).  Like the pack counter: one copy
// per device, its address looked up once per device, and the calls that use
// it serialised by g_pack_mu and synchronised before they return.
struct ConvScratch {
    uint32_t digits[bitnet::kConvPartials * bitnet::kConvDigits];   // AbsMean partial sums
    double partial[bitnet::kConvPartials];                          // max|w| per workgroup
    float alpha;
    unsigned bad;
    float wmax;
};
__device__ ConvScratch g_conv;
void *g_conv_addr[kMaxDevices];

int conv_scratch(const char *fn, ConvScratch **out) {
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return hip_fail(fn, e);
    if (dev < 0 || dev >= kMaxDevices)
        return fail(BITNET_E_HIP, "%s: device index %d unsupported", fn, dev);
    if (!g_conv_addr[dev]) {
        void *p = nullptr;
        e = hipGetSymbolAddress(&p, HIP_SYMBOL(g_conv));
        if (e != hipSuccess) return hip_fail(fn, e);
        g_conv_addr[dev] = p;
    }
    *out = static_cast<ConvScratch *>(g_conv_addr[dev]);
    return BITNET_OK;
}

int check_matmul(const char *fn, const uint8_t *packed, int64_t M, int64_t K,
                 const int8_t *xq, const float *xs, const int32_t *xsum, int64_t N,
                 int64_t max_n, const int32_t *dot, const float *y) {
    if (M < 0 || N < 0)
        return fail(BITNET_E_SHAPE, "%s: negative size M=%lld N=%lld", fn, (long long)M,
                    (long long)N);
    if (M > 0x7fffffffLL)
        return fail(BITNET_E_SHAPE, "%s: M=%lld exceeds 2^31-1", fn, (long long)M);
    if (N > max_n)
        return fail(BITNET_E_SHAPE, "%s: N=%lld exceeds %lld", fn, (long long)N,
                    (long long)max_n);
    if (int s = check_k(fn, K)) return s;
    if (M == 0 || N == 0) return BITNET_OK;
    if (!packed || !xq || !xs || !xsum)
        return fail(BITNET_E_NULL, "%s: packed, xq, x_scale and x_sum are required", fn);
    if (!dot && !y) return fail(BITNET_E_NULL, "%s: dot and y are both NULL", fn);
    if (!aligned(packed, 16) || !aligned(xq, 16))
        return fail(BITNET_E_ALIGN, "%s: packed and xq must be 16-byte aligned", fn);
    if (!aligned(xs, 4) || !aligned(xsum, 4) || (dot && !aligned(dot, 4)) ||
        (y && !aligned(y, 4)))
        return fail(BITNET_E_ALIGN, "%s: x_scale, x_sum, dot, y must be 4-byte aligned", fn);
    return BITNET_OK;
}

}  // namespace

BITNET_API int bitnet_abi_version(void) { return BITNET_ABI_VERSION; }

BITNET_API const char *bitnet_last_error(void) { return g_last_error.c_str(); }

BITNET_API int bitnet_pack_i2s(const int8_t *w, int64_t M, int64_t K, uint8_t *packed,
                               void *stream) {
    const char *fn = "bitnet_pack_i2s";
    if (M < 0) return fail(BITNET_E_SHAPE, "%s: negative M=%lld", fn, (long long)M);
    if (int s = check_k(fn, K)) return s;
    if (M == 0) return ok();
    if (!w || !packed) return fail(BITNET_E_NULL, "%s: w and packed are required", fn);
    if (!aligned(w, 4) || !aligned(packed, 16))
        return fail(BITNET_E_ALIGN, "%s: w must be 4-byte and packed 16-byte aligned", fn);
    hipStream_t st = static_cast<hipStream_t>(stream);
    std::lock_guard<std::mutex> lock(g_pack_mu);
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return hip_fail("bitnet_pack_i2s: hipGetDevice", e);
    unsigned *bad = nullptr;
    if (int s = pack_counter(dev, &bad)) return s;
    if ((e = hipMemsetAsync(bad, 0, sizeof(unsigned), st)) != hipSuccess)
        return hip_fail("bitnet_pack_i2s: clear counter", e);
    if ((e = bitnet::launch_pack(w, M, K, packed, bad, st)) != hipSuccess)
        return hip_fail("bitnet_pack_i2s: launch", e);
    unsigned nbad = 0;
    if ((e = hipMemcpyAsync(&nbad, bad, sizeof nbad, hipMemcpyDeviceToHost, st)) != hipSuccess)
        return hip_fail("bitnet_pack_i2s: read counter", e);
    if ((e = hipStreamSynchronize(st)) != hipSuccess)
        return hip_fail("bitnet_pack_i2s: synchronize", e);
    if (nbad)
        return fail(BITNET_E_VALUE, "%s: %u weight(s) outside {-1,0,+1}", fn, nbad);
    return ok();
}

BITNET_API int bitnet_absmean_i2s(const void *w, int dtype, int64_t M, int64_t K,
                                  uint8_t *packed, float *alpha, void *stream) {
    const char *fn = "bitnet_absmean_i2s";
    if (dtype != BITNET_F32 && dtype != BITNET_BF16)
        return fail(BITNET_E_DTYPE, "%s: unknown dtype %d", fn, dtype);
    if (M < 1) return fail(BITNET_E_SHAPE, "%s: M=%lld, need at least one row", fn, (long long)M);
    if (int s = check_k(fn, K)) return s;
    if (M > (1LL << 40) / K)
        return fail(BITNET_E_SHAPE, "%s: M*K exceeds 2^40 weights", fn);
    if (!w || !packed || !alpha) return fail(BITNET_E_NULL, "%s: w, packed and alpha are required", fn);
    if (!aligned(w, 16) || !aligned(packed, 16))
        return fail(BITNET_E_ALIGN, "%s: w and packed must be 16-byte aligned", fn);
    hipStream_t st = static_cast<hipStream_t>(stream);
    std::lock_guard<std::mutex> lock(g_pack_mu);
    ConvScratch *sc = nullptr;
    if (int s = conv_scratch(fn, &sc)) return s;
    hipError_t e = hipMemsetAsync(&sc->bad, 0, sizeof(unsigned), st);
    const int bf16 = dtype == BITNET_BF16;
    if (e == hipSuccess) e = bitnet::launch_absmean_alpha(w, bf16, M * K, sc->digits, &sc->alpha, st);
    if (e == hipSuccess)
        e = bitnet::launch_ternary_pack(w, bf16, 0, M, K, &sc->alpha, packed, &sc->bad, nullptr,
                                        nullptr, st);
    struct { float alpha; unsigned bad; } res{};
    if (e == hipSuccess) e = hipMemcpyAsync(&res, &sc->alpha, sizeof res, hipMemcpyDeviceToHost, st);
    if (e == hipSuccess) e = hipStreamSynchronize(st);
    if (e != hipSuccess) return hip_fail(fn, e);
    if (res.bad) return fail(BITNET_E_VALUE, "%s: %u non-finite weight(s)", fn, res.bad);
    *alpha = res.alpha;
    return ok();
}

BITNET_API int bitnet_pack_i2s_f32(const float *w, int64_t M, int64_t K, uint8_t *packed,
                                   float *w_max, void *stream) {
    const char *fn = "bitnet_pack_i2s_f32";
    if (M < 0) return fail(BITNET_E_SHAPE, "%s: negative M=%lld", fn, (long long)M);
    if (int s = check_k(fn, K)) return s;
    if (M == 0) {
        if (w_max) *w_max = 0.0f;
        return ok();
    }
    if (!w || !packed) return fail(BITNET_E_NULL, "%s: w and packed are required", fn);
    if (!aligned(w, 16) || !aligned(packed, 16))
        return fail(BITNET_E_ALIGN, "%s: w and packed must be 16-byte aligned", fn);
    hipStream_t st = static_cast<hipStream_t>(stream);
    std::lock_guard<std::mutex> lock(g_pack_mu);
    ConvScratch *sc = nullptr;
    if (int s = conv_scratch(fn, &sc)) return s;
    hipError_t e = hipMemsetAsync(&sc->bad, 0, sizeof(unsigned), st);
    if (e == hipSuccess)
        e = bitnet::launch_ternary_pack(w, 0, 1, M, K, nullptr, packed, &sc->bad, sc->partial,
                                        &sc->wmax, st);
    struct { unsigned bad; float wmax; } res{};
    if (e == hipSuccess) e = hipMemcpyAsync(&res, &sc->bad, sizeof res, hipMemcpyDeviceToHost, st);
    if (e == hipSuccess) e = hipStreamSynchronize(st);
    if (e != hipSuccess) return hip_fail(fn, e);
    if (res.bad) return fail(BITNET_E_VALUE, "%s: %u non-finite weight(s)", fn, res.bad);
    if (w_max) *w_max = res.wmax;
    return ok();
}

BITNET_API int bitnet_quant_act_i8(const void *x, int dtype, int64_t N, int64_t K, int8_t *xq,
                                   float *x_scale, int32_t *x_sum, void *stream) {
    const char *fn = "bitnet_quant_act_i8";
    if (dtype != BITNET_F32 && dtype != BITNET_BF16)
        return fail(BITNET_E_DTYPE, "%s: unknown dtype %d", fn, dtype);
    if (N < 0 || N > 0x7fffffffLL)
        return fail(BITNET_E_SHAPE, "%s: N=%lld out of range", fn, (long long)N);
    if (int s = check_k(fn, K)) return s;
    if (N == 0) return ok();
    if (!x || !xq || !x_scale || !x_sum)
        return fail(BITNET_E_NULL, "%s: x, xq, x_scale and x_sum are required", fn);
    if (!aligned(x, 16) || !aligned(xq, 16) || !aligned(x_scale, 4) || !aligned(x_sum, 4))
        return fail(BITNET_E_ALIGN, "%s: x and xq must be 16-byte aligned", fn);
    hipError_t e = bitnet::launch_quant(x, dtype == BITNET_BF16, N, K, xq, x_scale, x_sum,
                                        static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail("bitnet_quant_act_i8: launch", e);
    return ok();
}

BITNET_API int bitnet_gemv_i2s_i8(const uint8_t *packed, float w_scale, int64_t M, int64_t K,
                                  const int8_t *xq, const float *x_scale,
                                  const int32_t *x_sum, int64_t N, int32_t *dot, float *y,
                                  void *stream) {
    const char *fn = "bitnet_gemv_i2s_i8";
    if (int s = check_matmul(fn, packed, M, K, xq, x_scale, x_sum, N, BITNET_GEMV_MAX_N, dot, y))
        return s;
    if (M == 0 || N == 0) return ok();
    hipStream_t st = static_cast<hipStream_t>(stream);
    hipError_t e;
    if (N <= BITNET_VALU_MAX_N) {
        bitnet::GemvMat m{packed, dot, y, w_scale, (int)M, 0};
        e = bitnet::launch_gemv_valu(&m, 1, K, N, 0, xq, x_scale, x_sum, nullptr, nullptr,
                                     nullptr, st);
    } else {
        bitnet::GemmMat m{packed, dot, y, w_scale, (int)M, 0};
        e = bitnet::launch_gemv_mfma(&m, 1, K, xq, x_scale, x_sum, N, st);
    }
    if (e != hipSuccess) return hip_fail("bitnet_gemv_i2s_i8: launch", e);
    return ok();
}

BITNET_API int bitnet_gemv_i2s_lut(const uint8_t *packed, float w_scale, int64_t M, int64_t K,
                                   const int8_t *xq, const float *x_scale,
                                   const int32_t *x_sum, int64_t N, int32_t *dot, float *y,
                                   void *stream) {
    const char *fn = "bitnet_gemv_i2s_lut";
    if (int s = check_matmul(fn, packed, M, K, xq, x_scale, x_sum, N, BITNET_GEMV_MAX_N, dot, y))
        return s;
    if (K > BITNET_LUT_MAX_K)
        return fail(BITNET_E_SHAPE, "%s: K=%lld exceeds %d", fn, (long long)K, BITNET_LUT_MAX_K);
    if (M == 0 || N == 0) return ok();
    hipError_t e = bitnet::launch_gemv_lut(packed, w_scale, M, K, xq, x_scale, x_sum, N, dot, y,
                                           static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail("bitnet_gemv_i2s_lut: launch", e);
    return ok();
}

BITNET_API int bitnet_gemm_i2s_i8(const uint8_t *packed, float w_scale, int64_t M, int64_t K,
                                  const int8_t *xq, const float *x_scale,
                                  const int32_t *x_sum, int64_t N, int32_t *dot, float *y,
                                  void *stream) {
    const char *fn = "bitnet_gemm_i2s_i8";
    if (int s = check_matmul(fn, packed, M, K, xq, x_scale, x_sum, N, BITNET_GEMM_MAX_N, dot, y))
        return s;
    if (M == 0 || N == 0) return ok();
    const bitnet::GemmMat m{packed, dot, y, w_scale, (int)M, 0};
    hipError_t e = bitnet::launch_gemm_mfma(&m, 1, K, xq, x_scale, x_sum, N,
                                            static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail("bitnet_gemm_i2s_i8: launch", e);
    return ok();
}

// Validate a host array of matrix descriptors (shared by the grouped calls).
static int check_mats(const char *fn, const bitnet_i2s_matrix *mats, int n_mats) {
    if (n_mats < 1 || n_mats > BITNET_MAX_GROUP)
        return fail(BITNET_E_SHAPE, "%s: n_mats=%d outside [1, %d]", fn, n_mats,
                    BITNET_MAX_GROUP);
    if (!mats) return fail(BITNET_E_NULL, "%s: mats is NULL", fn);
    for (int i = 0; i < n_mats; ++i) {
        const bitnet_i2s_matrix &m = mats[i];
        if (m.M < 0 || m.M > 0x7fffffffLL)
            return fail(BITNET_E_SHAPE, "%s: mats[%d].M=%lld out of range", fn, i, (long long)m.M);
        if (m.M > 0) {
            if (!m.packed) return fail(BITNET_E_NULL, "%s: mats[%d].packed is NULL", fn, i);
            if (!m.dot && !m.y)
                return fail(BITNET_E_NULL, "%s: mats[%d] has neither dot nor y", fn, i);
            if (!aligned(m.packed, 16))
                return fail(BITNET_E_ALIGN, "%s: mats[%d].packed must be 16-byte aligned", fn, i);
            if ((m.dot && !aligned(m.dot, 4)) || (m.y && !aligned(m.y, 4)))
                return fail(BITNET_E_ALIGN, "%s: mats[%d] outputs must be 4-byte aligned", fn, i);
        }
    }
    return BITNET_OK;
}

BITNET_API int bitnet_ffn_act_quant_i8(const float *g, const float *u, const float *gamma,
                                      float eps, int64_t N, int64_t F, int8_t *xq,
                                      float *x_scale, int32_t *x_sum, void *stream) {
    const char *fn = "bitnet_ffn_act_quant_i8";
    if (N < 0) return fail(BITNET_E_SHAPE, "%s: negative N=%lld", fn, (long long)N);
    if (N > 0x7fffffffLL) return fail(BITNET_E_SHAPE, "%s: N=%lld exceeds 2^31-1", fn, (long long)N);
    if (int s = check_k(fn, F)) return s;
    if (!(eps > 0.0f) || !(eps < 3.4e38f))
        return fail(BITNET_E_VALUE, "%s: eps must be positive and finite", fn);
    if (N == 0) return ok();
    if (!g || !u || !xq || !x_scale || !x_sum)
        return fail(BITNET_E_NULL, "%s: g, u, xq, x_scale and x_sum are required", fn);
    if (!aligned(g, 16) || !aligned(u, 16) || (gamma && !aligned(gamma, 16)) ||
        !aligned(xq, 16) || !aligned(x_scale, 4) || !aligned(x_sum, 4))
        return fail(BITNET_E_ALIGN, "%s: g, u, gamma and xq must be 16-byte aligned", fn);
    hipError_t e = bitnet::launch_ffn_act_quant(g, u, gamma, eps, N, F, xq, x_scale, x_sum,
                                                static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(fn, e);
    return ok();
}

BITNET_API int bitnet_gemv_i2s_i8_group(const bitnet_i2s_matrix *mats, int n_mats, int64_t K,
                                        const int8_t *xq, const float *x_scale,
                                        const int32_t *x_sum, int64_t N, void *stream) {
    const char *fn = "bitnet_gemv_i2s_i8_group";
    if (int s = check_mats(fn, mats, n_mats)) return s;
    if (N < 0 || N > BITNET_GEMV_MAX_N)
        return fail(BITNET_E_SHAPE, "%s: N=%lld outside [0, %d]", fn, (long long)N,
                    BITNET_GEMV_MAX_N);
    if (int s = check_k(fn, K)) return s;
    int64_t rows = 0;
    for (int i = 0; i < n_mats; ++i) rows += mats[i].M;
    if (N == 0 || rows == 0) return ok();
    if (!xq || !x_scale || !x_sum)
        return fail(BITNET_E_NULL, "%s: xq, x_scale and x_sum are required", fn);
    if (!aligned(xq, 16) || !aligned(x_scale, 4) || !aligned(x_sum, 4))
        return fail(BITNET_E_ALIGN, "%s: xq must be 16-byte and x_scale/x_sum 4-byte aligned", fn);
    hipStream_t st = static_cast<hipStream_t>(stream);
    hipError_t e = hipSuccess;
    if (N <= BITNET_VALU_MAX_N) {
        bitnet::GemvMat gm[bitnet::kMaxMats];
        for (int i = 0; i < n_mats; ++i)
            gm[i] = bitnet::GemvMat{mats[i].packed, mats[i].dot, mats[i].y, mats[i].w_scale,
                                    (int)mats[i].M, 0};
        e = bitnet::launch_gemv_valu(gm, n_mats, K, N, 0, xq, x_scale, x_sum, nullptr, nullptr,
                                     nullptr, st);
    } else {
        bitnet::GemmMat mm[bitnet::kMaxMats];
        for (int i = 0; i < n_mats; ++i)
            mm[i] = bitnet::GemmMat{mats[i].packed, mats[i].dot, mats[i].y, mats[i].w_scale,
                                    (int)mats[i].M, 0};
        e = bitnet::launch_gemv_mfma(mm, n_mats, K, xq, x_scale, x_sum, N, st);
    }
    if (e != hipSuccess) return hip_fail(fn, e);
    return ok();
}

BITNET_API int bitnet_gemm_i2s_i8_group(const bitnet_i2s_matrix *mats, int n_mats, int64_t K,
                                        const int8_t *xq, const float *x_scale,
                                        const int32_t *x_sum, int64_t N, void *stream) {
    const char *fn = "bitnet_gemm_i2s_i8_group";
    if (int s = check_mats(fn, mats, n_mats)) return s;
    if (N < 0 || N > BITNET_GEMM_MAX_N)
        return fail(BITNET_E_SHAPE, "%s: N=%lld outside [0, %d]", fn, (long long)N,
                    BITNET_GEMM_MAX_N);
    if (int s = check_k(fn, K)) return s;
    bitnet::GemmMat gm[bitnet::kMaxMats];
    int64_t rows = 0;
    for (int i = 0; i < n_mats; ++i) {
        gm[i] = bitnet::GemmMat{mats[i].packed, mats[i].dot, mats[i].y, mats[i].w_scale,
                                (int)mats[i].M, 0};
        rows += mats[i].M;
    }
    if (N == 0 || rows == 0) return ok();
    if (!xq || !x_scale || !x_sum)
        return fail(BITNET_E_NULL, "%s: xq, x_scale and x_sum are required", fn);
    if (!aligned(xq, 16) || !aligned(x_scale, 4) || !aligned(x_sum, 4))
        return fail(BITNET_E_ALIGN, "%s: xq must be 16-byte and x_scale/x_sum 4-byte aligned", fn);
    hipError_t e = bitnet::launch_gemm_mfma(gm, n_mats, K, xq, x_scale, x_sum, N,
                                            static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(fn, e);
    return ok();
}

static int linear_impl(const char *fn, const void *x, int dtype, int64_t N, int64_t K,
                       const bitnet_i2s_matrix *mats, int n_mats, int8_t *xq, float *x_scale,
                       int32_t *x_sum, void *stream) {
    if (dtype != BITNET_F32 && dtype != BITNET_BF16)
        return fail(BITNET_E_DTYPE, "%s: unknown dtype %d", fn, dtype);
    if (N < 0 || N > BITNET_GEMM_MAX_N)
        return fail(BITNET_E_SHAPE, "%s: N=%lld outside [0, %d]", fn, (long long)N,
                    BITNET_GEMM_MAX_N);
    if (int s = check_k(fn, K)) return s;
    if (int s = check_mats(fn, mats, n_mats)) return s;
    bitnet::GemvMat gm[bitnet::kMaxMats];
    for (int i = 0; i < n_mats; ++i)
        gm[i] = bitnet::GemvMat{mats[i].packed, mats[i].dot, mats[i].y, mats[i].w_scale,
                                (int)mats[i].M, 0};
    if (N == 0) return ok();
    if (!x) return fail(BITNET_E_NULL, "%s: x is NULL", fn);
    if (!aligned(x, 16) || (xq && !aligned(xq, 16)) || (x_scale && !aligned(x_scale, 4)) ||
        (x_sum && !aligned(x_sum, 4)))
        return fail(BITNET_E_ALIGN, "%s: x/xq must be 16-byte and x_scale/x_sum 4-byte aligned", fn);
    if (N > BITNET_LINEAR_FUSED_MAX_N && (!xq || !x_scale || !x_sum))
        return fail(BITNET_E_NULL, "%s: N > %d needs the xq, x_scale and x_sum buffers", fn,
                    BITNET_LINEAR_FUSED_MAX_N);
    hipStream_t st = static_cast<hipStream_t>(stream);
    hipError_t e;
    if (N <= BITNET_LINEAR_FUSED_MAX_N) {
        e = bitnet::launch_gemv_valu(gm, n_mats, K, N, dtype == BITNET_BF16 ? 2 : 1, x, nullptr,
                                     nullptr, xq, x_scale, x_sum, st);
    } else if (N <= BITNET_GEMV_MAX_N) {
        e = bitnet::launch_quant(x, dtype == BITNET_BF16, N, K, xq, x_scale, x_sum, st);
        if (e == hipSuccess) {
            bitnet::GemmMat mm[bitnet::kMaxMats];
            for (int i = 0; i < n_mats; ++i)
                mm[i] = bitnet::GemmMat{gm[i].packed, gm[i].dot, gm[i].y, gm[i].alpha, gm[i].M, 0};
            e = bitnet::launch_gemv_mfma(mm, n_mats, K, xq, x_scale, x_sum, N, st);
        }
    } else {
        e = bitnet::launch_quant(x, dtype == BITNET_BF16, N, K, xq, x_scale, x_sum, st);
        if (e == hipSuccess) {
            bitnet::GemmMat mm[bitnet::kMaxMats];
            for (int i = 0; i < n_mats; ++i)
                mm[i] = bitnet::GemmMat{gm[i].packed, gm[i].dot, gm[i].y, gm[i].alpha, gm[i].M, 0};
            e = bitnet::launch_gemm_mfma(mm, n_mats, K, xq, x_scale, x_sum, N, st);
        }
    }
    if (e != hipSuccess) return hip_fail(fn, e);
    return ok();
}

BITNET_API int bitnet_linear_i2s(const void *x, int dtype, int64_t N, int64_t K,
                                 const bitnet_i2s_matrix *mats, int n_mats, int8_t *xq,
                                 float *x_scale, int32_t *x_sum, void *stream) {
    return linear_impl("bitnet_linear_i2s", x, dtype, N, K, mats, n_mats, xq, x_scale, x_sum,
                       stream);
}

BITNET_API int bitnet_block_norm_quant_i8(const void *b, int b_dtype, int post,
                                          const float *post_gamma, const float *gate,
                                          int64_t gate_stride, float scale, const void *res,
                                          void *h, int dtype, const float *gamma, float eps,
                                          int64_t N, int64_t F, void *v, int8_t *xq,
                                          float *x_scale, int32_t *x_sum, void *stream) {
    const char *fn = "bitnet_block_norm_quant_i8";
    for (int d : {b_dtype, dtype})
        if (d != BITNET_F32 && d != BITNET_BF16)
            return fail(BITNET_E_DTYPE, "%s: unknown dtype %d", fn, d);
    if (N < 0 || N > 0x7fffffffLL)
        return fail(BITNET_E_SHAPE, "%s: N=%lld out of range", fn, (long long)N);
    if (int s = check_k(fn, F)) return s;
    if (!(eps > 0.0f) || !(eps < 3.4e38f))
        return fail(BITNET_E_VALUE, "%s: eps must be positive and finite", fn);
    if (!(scale > -3.4e38f) || !(scale < 3.4e38f))
        return fail(BITNET_E_VALUE, "%s: scale must be finite", fn);
    if (gate && gate_stride != 0 && (gate_stride < F || gate_stride % 4 != 0))
        return fail(BITNET_E_SHAPE, "%s: gate_stride=%lld must be 0 or a multiple of 4, at least F",
                    fn, (long long)gate_stride);
    if (N == 0) return ok();
    if (!b) return fail(BITNET_E_NULL, "%s: b is required", fn);
    if (h && !res) return fail(BITNET_E_NULL, "%s: h without res", fn);
    if (post_gamma && !post) return fail(BITNET_E_VALUE, "%s: post_gamma without post", fn);
    if ((xq || x_scale || x_sum) && !(xq && x_scale && x_sum))
        return fail(BITNET_E_NULL, "%s: xq, x_scale and x_sum come together", fn);
    if (!h && !v && !xq) return fail(BITNET_E_NULL, "%s: h, v and xq are all NULL", fn);
    for (const void *p : {b, (const void *)post_gamma, (const void *)gate, res, (const void *)h,
                          (const void *)gamma, (const void *)v, (const void *)xq})
        if (!aligned(p, 16))
            return fail(BITNET_E_ALIGN, "%s: rows and gains must be 16-byte aligned", fn);
    if (!aligned(x_scale, 4) || !aligned(x_sum, 4))
        return fail(BITNET_E_ALIGN, "%s: x_scale and x_sum must be 4-byte aligned", fn);
    const bitnet::BlockNormArgs a{b, post_gamma, gate, gamma, res, h, v, xq, x_scale, x_sum,
                                  gate_stride, scale, eps, (int)F, post != 0};
    hipError_t e = bitnet::launch_block_norm(a, N, b_dtype == BITNET_BF16, dtype == BITNET_BF16,
                                             static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(fn, e);
    return ok();
}

// Validate a cache descriptor and a call's row count (shared by the cache calls).
static int check_kv4(const char *fn, const bitnet_kv4_batch *c, int dtype, int64_t N,
                     bool rows = true) {
    if (!c) return fail(BITNET_E_NULL, "%s: batch is NULL", fn);
    if (dtype != BITNET_F32 && dtype != BITNET_BF16)
        return fail(BITNET_E_DTYPE, "%s: unknown dtype %d", fn, dtype);
    if (N < 0 || N > BITNET_GEMM_MAX_N)
        return fail(BITNET_E_SHAPE, "%s: N=%lld outside [0, %d]", fn, (long long)N,
                    BITNET_GEMM_MAX_N);
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
        return fail(BITNET_E_SHAPE, "%s: head_dim=%lld must be 64, 128 or 256", fn,
                    (long long)c->head_dim);
    if (c->n_kv_heads < 1 || c->n_kv_heads > BITNET_KV4_MAX_HEADS)
        return fail(BITNET_E_SHAPE, "%s: n_kv_heads=%lld outside [1, %d]", fn,
                    (long long)c->n_kv_heads, BITNET_KV4_MAX_HEADS);
    if (c->n_pages < 1 || c->n_pages > 0x7fffffffLL)
        return fail(BITNET_E_SHAPE, "%s: n_pages=%lld out of range", fn, (long long)c->n_pages);
    if (c->max_pages < 1 || c->max_pages > BITNET_KV4_MAX_PAGES)
        return fail(BITNET_E_SHAPE, "%s: max_pages=%lld outside [1, %d]", fn,
                    (long long)c->max_pages, BITNET_KV4_MAX_PAGES);
    if (c->n_seqs < 0 || c->n_seqs > BITNET_KV4_MAX_SEQS)
        return fail(BITNET_E_SHAPE, "%s: n_seqs=%lld outside [0, %d]", fn, (long long)c->n_seqs,
                    BITNET_KV4_MAX_SEQS);
    if (N == 0 || c->n_seqs == 0) return BITNET_OK;
    if (!c->cache || !c->table || !c->kv_len || (rows && !c->q_start))
        return fail(BITNET_E_NULL, "%s: cache, table, kv_len and q_start are required", fn);
    if (!aligned(c->cache, 16))
        return fail(BITNET_E_ALIGN, "%s: cache must be 16-byte aligned", fn);
    if (!aligned(c->table, 4) || !aligned(c->kv_len, 4) || (rows && !aligned(c->q_start, 4)))
        return fail(BITNET_E_ALIGN, "%s: table, kv_len and q_start must be 4-byte aligned", fn);
    return BITNET_OK;
}

// A [N] row array of heads * dim values with a stride, in elements.
static int check_rows(const char *fn, const char *name, const void *p, int64_t stride, int64_t row,
                      int dtype) {
    const int64_t per16 = dtype == BITNET_BF16 ? 8 : 4;
    if (!p) return fail(BITNET_E_NULL, "%s: %s is required", fn, name);
    if (stride < row || stride % per16 != 0 || stride > (1LL << 40))
        return fail(BITNET_E_SHAPE, "%s: %s_stride=%lld must be a multiple of %lld and at least %lld",
                    fn, name, (long long)stride, (long long)per16, (long long)row);
    if (!aligned(p, 16)) return fail(BITNET_E_ALIGN, "%s: %s must be 16-byte aligned", fn, name);
    return BITNET_OK;
}

static bitnet::Kv4Args kv4_args(const bitnet_kv4_batch *c) {
    return bitnet::Kv4Args{static_cast<uint8_t *>(c->cache), c->table, c->kv_len, c->q_start,
                           c->n_pages, c->max_pages, c->n_seqs, (int)c->n_kv_heads};
}

BITNET_API int bitnet_kv4_append(const bitnet_kv4_batch *batch, const void *k, int64_t k_stride,
                                 const void *v, int64_t v_stride, int dtype, int64_t N,
                                 void *stream) {
    const char *fn = "bitnet_kv4_append";
    if (int s = check_kv4(fn, batch, dtype, N)) return s;
    if (N == 0 || batch->n_seqs == 0) return ok();
    const int64_t row = batch->n_kv_heads * batch->head_dim;
    if (int s = check_rows(fn, "k", k, k_stride, row, dtype)) return s;
    if (int s = check_rows(fn, "v", v, v_stride, row, dtype)) return s;
    hipError_t e = bitnet::launch_kv4_append(kv4_args(batch), k, v, dtype == BITNET_BF16, k_stride,
                                             v_stride, N, (int)batch->head_dim,
                                             static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(fn, e);
    return ok();
}

BITNET_API int bitnet_kv4_read(const bitnet_kv4_batch *batch, void *k, void *v, int dtype,
                               int64_t N, void *stream) {
    const char *fn = "bitnet_kv4_read";
    if (int s = check_kv4(fn, batch, dtype, N)) return s;
    if (N == 0 || batch->n_seqs == 0) return ok();
    if (!k && !v) return fail(BITNET_E_NULL, "%s: k and v are both NULL", fn);
    if (!aligned(k, 16) || !aligned(v, 16))
        return fail(BITNET_E_ALIGN, "%s: k and v must be 16-byte aligned", fn);
    hipError_t e = bitnet::launch_kv4_read(kv4_args(batch), k, v, dtype == BITNET_BF16, N,
                                           (int)batch->head_dim, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(fn, e);
    return ok();
}

static int check_heads(const char *fn, int64_t heads, int64_t kv_heads) {
    if (heads < 1 || heads > BITNET_KV4_MAX_HEADS || kv_heads < 1 || heads % kv_heads != 0)
        return fail(BITNET_E_SHAPE, "%s: n_heads=%lld must be a multiple of n_kv_heads=%lld, at most %d",
                    fn, (long long)heads, (long long)kv_heads, BITNET_KV4_MAX_HEADS);
    return BITNET_OK;
}

BITNET_API int64_t bitnet_attn_kv4_workspace(int64_t n_seqs, int64_t N, int64_t n_heads,
                                             int64_t n_kv_heads, int64_t head_dim,
                                             int64_t max_kv, int64_t window, int64_t sinks) {
    const char *fn = "bitnet_attn_kv4_workspace";
    if (check_heads(fn, n_heads, n_kv_heads)) return -1;
    if (n_seqs < 0 || n_seqs > BITNET_KV4_MAX_SEQS || N < 0 || N > BITNET_GEMM_MAX_N ||
        max_kv < 0 || max_kv > (int64_t)BITNET_KV4_MAX_PAGES * BITNET_KV4_PAGE || window < 0 ||
        window > 0x7fffffffLL || sinks < 0 || sinks > 0x7fffffffLL ||
        (head_dim != 64 && head_dim != 128 && head_dim != 256)) {
        fail(BITNET_E_SHAPE, "%s: sizes out of range", fn);
        return -1;
    }
    g_last_error.clear();
    if (n_seqs == 0 || N == 0) return 0;
    int64_t splits = 1;   // the larger of the two types
    for (bool bf16 : {false, true}) {
        const bitnet::Attn4Plan p = bitnet::attn4_plan(n_seqs, N, n_heads, n_kv_heads, head_dim,
                                                       max_kv, window, sinks, bf16);
        if (p.workgroups >= bitnet::kAttn4Workgroups) {
            fail(BITNET_E_SHAPE, "%s: N=%lld, n_seqs=%lld are too many rows for one call", fn,
                 (long long)N, (long long)n_seqs);
            return -1;
        }
        splits = std::max<int64_t>(splits, p.splits);
    }
    return splits > 1 ? splits * N * n_heads * (head_dim + 4) * 4 : 0;
}

BITNET_API int bitnet_attn_kv4(const bitnet_kv4_batch *batch, const void *q, int64_t q_stride,
                               int dtype, int64_t N, int64_t n_heads, float scale, int64_t window,
                               int64_t sinks, int64_t max_kv, void *out, void *workspace,
                               int64_t workspace_bytes, void *stream) {
    const char *fn = "bitnet_attn_kv4";
    if (int s = check_kv4(fn, batch, dtype, N)) return s;
    if (int s = check_heads(fn, n_heads, batch->n_kv_heads)) return s;
    if (!(scale > 0.0f) || !(scale < 3.4e38f))
        return fail(BITNET_E_VALUE, "%s: scale must be positive and finite", fn);
    if (window < 0 || sinks < 0 || window > 0x7fffffffLL || sinks > 0x7fffffffLL)
        return fail(BITNET_E_SHAPE, "%s: window=%lld, sinks=%lld out of range", fn,
                    (long long)window, (long long)sinks);
    if (max_kv < 0 || max_kv > batch->max_pages * BITNET_KV4_PAGE)
        return fail(BITNET_E_SHAPE, "%s: max_kv=%lld outside [0, 64 * max_pages]", fn,
                    (long long)max_kv);
    if (N == 0 || batch->n_seqs == 0) return ok();
    if (int s = check_rows(fn, "q", q, q_stride, n_heads * batch->head_dim, dtype)) return s;
    if (!out) return fail(BITNET_E_NULL, "%s: out is required", fn);
    if (!aligned(out, 16) || !aligned(workspace, 16))
        return fail(BITNET_E_ALIGN, "%s: out and workspace must be 16-byte aligned", fn);
    const int64_t need = bitnet_attn_kv4_workspace(batch->n_seqs, N, n_heads, batch->n_kv_heads,
                                                   batch->head_dim, max_kv, window, sinks);
    if (need < 0) return BITNET_E_SHAPE;   // it has said why
    if (need > 0 && !workspace)
        return fail(BITNET_E_NULL, "%s: a workspace of %lld bytes is required", fn, (long long)need);
    if (workspace_bytes < need)
        return fail(BITNET_E_SHAPE, "%s: the workspace has %lld bytes, %lld are required", fn,
                    (long long)workspace_bytes, (long long)need);
    // positions stay below 2^30, so no window or sink beyond says more
    const int far = 1 << 30, win = (int)(window < far ? window : far);
    const int first = (int)(sinks < far ? sinks : far);
    const bitnet::Attn4Plan sp =
        bitnet::attn4_plan(batch->n_seqs, N, n_heads, batch->n_kv_heads, batch->head_dim, max_kv,
                           window, sinks, dtype == BITNET_BF16);
    const bitnet::Attn4Args a{kv4_args(batch), q, out, static_cast<float *>(workspace), q_stride, N,
                              scale * 1.4426950408889634f, (int)n_heads, win, first, sp.splits,
                              (uint32_t)sp.tiles};
    hipError_t e = bitnet::launch_attn4(a, sp, dtype == BITNET_BF16, (int)batch->head_dim,
                                        static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(fn, e);
    return ok();
}

BITNET_API int64_t bitnet_kv4_weigh_workspace(int64_t n_seqs, int64_t N, int64_t n_heads,
                                              int64_t n_kv_heads, int64_t head_dim,
                                              int64_t max_kv, int64_t window, int64_t sinks) {
    const char *fn = "bitnet_kv4_weigh_workspace";
    if (check_heads(fn, n_heads, n_kv_heads)) return -1;
    if (n_seqs < 0 || n_seqs > BITNET_KV4_MAX_SEQS || N < 0 || N > BITNET_GEMM_MAX_N ||
        max_kv < 0 || max_kv > (int64_t)BITNET_KV4_MAX_PAGES * BITNET_KV4_PAGE || window < 0 ||
        window > 0x7fffffffLL || sinks < 0 || sinks > 0x7fffffffLL ||
        (head_dim != 64 && head_dim != 128 && head_dim != 256)) {
        fail(BITNET_E_SHAPE, "%s: sizes out of range", fn);
        return -1;
    }
    g_last_error.clear();
    if (n_seqs == 0 || N == 0) return 0;
    // of the two types, fp32 takes the more
    return bitnet::weigh_plan(n_seqs, N, n_heads, n_kv_heads, head_dim, max_kv, window, sinks, false)
        .bytes;
}

BITNET_API int bitnet_kv4_weigh(const bitnet_kv4_batch *batch, const void *q, int64_t q_stride,
                                int dtype, int64_t N, int64_t n_heads, float scale, int64_t window,
                                int64_t sinks, int64_t max_kv, const float *weights, float decay,
                                float *out, void *workspace, int64_t workspace_bytes,
                                void *stream) {
    const char *fn = "bitnet_kv4_weigh";
    if (int s = check_kv4(fn, batch, dtype, N)) return s;
    if (int s = check_heads(fn, n_heads, batch->n_kv_heads)) return s;
    if (!(scale > 0.0f) || !(scale < 3.4e38f))
        return fail(BITNET_E_VALUE, "%s: scale must be positive and finite", fn);
    if (!(decay >= 0.0f) || !(decay < 3.4e38f))
        return fail(BITNET_E_VALUE, "%s: decay must be finite and not negative", fn);
    if (window < 0 || sinks < 0 || window > 0x7fffffffLL || sinks > 0x7fffffffLL)
        return fail(BITNET_E_SHAPE, "%s: window=%lld, sinks=%lld out of range", fn,
                    (long long)window, (long long)sinks);
    if (max_kv < 0 || max_kv > batch->max_pages * BITNET_KV4_PAGE)
        return fail(BITNET_E_SHAPE, "%s: max_kv=%lld outside [0, 64 * max_pages]", fn,
                    (long long)max_kv);
    if (N == 0 || batch->n_seqs == 0) return ok();
    if (int s = check_rows(fn, "q", q, q_stride, n_heads * batch->head_dim, dtype)) return s;
    if (!out || (!weights && decay != 0.0f))
        return fail(BITNET_E_NULL, "%s: out, and weights with a decay, are required", fn);
    if (!aligned(out, 16) || !aligned(weights, 16) || !aligned(workspace, 16))
        return fail(BITNET_E_ALIGN, "%s: weights, out and workspace must be 16-byte aligned", fn);
    const bitnet::WeighPlan p =
        bitnet::weigh_plan(batch->n_seqs, N, n_heads, batch->n_kv_heads, batch->head_dim, max_kv,
                           window, sinks, dtype == BITNET_BF16);
    const int64_t need = bitnet_kv4_weigh_workspace(batch->n_seqs, N, n_heads, batch->n_kv_heads,
                                                    batch->head_dim, max_kv, window, sinks);
    if (!workspace)
        return fail(BITNET_E_NULL, "%s: a workspace of %lld bytes is required", fn, (long long)need);
    if (workspace_bytes < need)
        return fail(BITNET_E_SHAPE, "%s: the workspace has %lld bytes, %lld are required", fn,
                    (long long)workspace_bytes, (long long)need);
    const int far = 1 << 30, win = (int)(window < far ? window : far);   // as bitnet_attn_kv4
    char *const ws = static_cast<char *>(workspace);
    const bitnet::WeighArgs a{kv4_args(batch), q, weights, out, reinterpret_cast<float2 *>(ws),
                              p.many ? reinterpret_cast<uint4 *>(ws + p.kept_at) : nullptr,
                              reinterpret_cast<float *>(ws + p.sums_at), q_stride, N, scale * 1.4426950408889634f, decay, (int)n_heads, win,
                              (int)(sinks < far ? sinks : far), p.splits};
    hipError_t e = bitnet::launch_kv4_weigh(a, p, dtype == BITNET_BF16, (int)batch->head_dim,
                                            static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(fn, e);
    return ok();
}

BITNET_API int64_t bitnet_kv4_evict_workspace(int64_t n_seqs, int64_t n_kv_heads,
                                              int64_t max_pages) {
    const char *fn = "bitnet_kv4_evict_workspace";
    if (n_seqs < 0 || n_seqs > BITNET_KV4_MAX_SEQS || n_kv_heads < 1 ||
        n_kv_heads > BITNET_KV4_MAX_HEADS || max_pages < 1 || max_pages > BITNET_KV4_MAX_PAGES) {
        fail(BITNET_E_SHAPE, "%s: sizes out of range", fn);
        return -1;
    }
    g_last_error.clear();
    return n_seqs ? bitnet::evict_plan(n_seqs, n_kv_heads, max_pages).bytes : 0;
}

BITNET_API int bitnet_kv4_evict(const bitnet_kv4_batch *batch, float *weights,
                                const int32_t *new_table, int64_t new_max_pages, int64_t keep,
                                int64_t sinks, int64_t recent, int32_t *new_len, int32_t *index,
                                void *workspace, int64_t workspace_bytes, void *stream) {
    const char *fn = "bitnet_kv4_evict";
    if (int s = check_kv4(fn, batch, BITNET_F32, 1, false)) return s;
    if (new_max_pages < 1 || new_max_pages > BITNET_KV4_MAX_PAGES)
        return fail(BITNET_E_SHAPE, "%s: new_max_pages=%lld outside [1, %d]", fn,
                    (long long)new_max_pages, BITNET_KV4_MAX_PAGES);
    if (keep < 1 || keep > new_max_pages * BITNET_KV4_PAGE)
        return fail(BITNET_E_SHAPE, "%s: keep=%lld outside [1, 64 * new_max_pages]", fn,
                    (long long)keep);
    if (sinks < 0 || recent < 0 || sinks > keep || recent > keep - sinks)
        return fail(BITNET_E_SHAPE, "%s: sinks=%lld and recent=%lld are more than keep=%lld", fn,
                    (long long)sinks, (long long)recent, (long long)keep);
    if (batch->n_seqs == 0) return ok();
    if (!weights || !new_table || !new_len || !index)
        return fail(BITNET_E_NULL, "%s: weights, new_table, new_len and index are required", fn);
    if (!aligned(weights, 16) || !aligned(workspace, 16))
        return fail(BITNET_E_ALIGN, "%s: weights and workspace must be 16-byte aligned", fn);
    if (!aligned(new_table, 4) || !aligned(new_len, 4) || !aligned(index, 4))
        return fail(BITNET_E_ALIGN, "%s: new_table, new_len and index must be 4-byte aligned", fn);
    const bitnet::EvictPlan p =
        bitnet::evict_plan(batch->n_seqs, batch->n_kv_heads, batch->max_pages);
    if (p.bytes > 0 && !workspace)
        return fail(BITNET_E_NULL, "%s: a workspace of %lld bytes is required", fn,
                    (long long)p.bytes);
    if (workspace_bytes < p.bytes)
        return fail(BITNET_E_SHAPE, "%s: the workspace has %lld bytes, %lld are required", fn,
                    (long long)workspace_bytes, (long long)p.bytes);
    // heads that have not begun still read the old lengths
    if (new_len < batch->kv_len + batch->n_seqs && batch->kv_len < new_len + batch->n_seqs)
        return fail(BITNET_E_VALUE, "%s: new_len overlaps kv_len", fn);
    if (new_table == batch->table)
        return fail(BITNET_E_VALUE, "%s: new_table is table", fn);
    char *const ws = static_cast<char *>(workspace);
    const bitnet::EvictArgs a{static_cast<uint8_t *>(batch->cache), weights, batch->table,
                              batch->kv_len, new_table, new_len, index,
                              reinterpret_cast<int *>(ws), reinterpret_cast<int2 *>(ws + p.search_at),
                              reinterpret_cast<int2 *>(ws + p.slices_at), batch->n_pages,
                              batch->max_pages, new_max_pages, batch->n_seqs,
                              (int)batch->n_kv_heads, (int)keep, (int)sinks, (int)recent};
    hipError_t e = bitnet::launch_kv4_evict(a, p, (int)batch->head_dim,
                                            static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(fn, e);
    return ok();
}

static int check_plan(const char *fn, const bitnet_rotary_plan *p, int64_t dim) {
    if (!p) return fail(BITNET_E_NULL, "%s: plan is NULL", fn);
    if (p->rot < 2 || p->rot > dim || p->rot % 2 != 0)
        return fail(BITNET_E_SHAPE, "%s: rot=%lld must be even and in [2, %lld]", fn,
                    (long long)p->rot, (long long)dim);
    if (!(p->magnitude > 0.0) || !(p->magnitude < 1e30))
        return fail(BITNET_E_VALUE, "%s: magnitude must be positive and finite", fn);
    return BITNET_OK;
}
static int check_turns(const char *fn, const bitnet_rotary_plan *p) {
    if (!p->turns) return fail(BITNET_E_NULL, "%s: turns is NULL", fn);
    if (!aligned(p->turns, 8)) return fail(BITNET_E_ALIGN, "%s: turns must be 8-byte aligned", fn);
    return BITNET_OK;
}

BITNET_API int bitnet_rotary(const bitnet_rotary_plan *plan, const void *x, int64_t x_stride,
                             int dtype, int64_t N, int64_t n_heads, int64_t head_dim,
                             const int32_t *positions, int inverse, void *out, int64_t out_stride,
                             void *stream) {
    const char *fn = "bitnet_rotary";
    if (dtype != BITNET_F32 && dtype != BITNET_BF16)
        return fail(BITNET_E_DTYPE, "%s: unknown dtype %d", fn, dtype);
    if (N < 0 || N > BITNET_GEMM_MAX_N)
        return fail(BITNET_E_SHAPE, "%s: N=%lld outside [0, %d]", fn, (long long)N,
                    BITNET_GEMM_MAX_N);
    if (head_dim < 8 || head_dim > BITNET_ROTARY_MAX_DIM || head_dim % 8 != 0)
        return fail(BITNET_E_SHAPE, "%s: head_dim=%lld must be a multiple of 8, at most %d", fn,
                    (long long)head_dim, BITNET_ROTARY_MAX_DIM);
    if (n_heads < 1 || n_heads > BITNET_KV4_MAX_HEADS)
        return fail(BITNET_E_SHAPE, "%s: n_heads=%lld outside [1, %d]", fn, (long long)n_heads,
                    BITNET_KV4_MAX_HEADS);
    if (int s = check_plan(fn, plan, head_dim)) return s;
    if (N == 0) return ok();
    if (int s = check_turns(fn, plan)) return s;
    const int64_t row = n_heads * head_dim;
    if (int s = check_rows(fn, "x", x, x_stride, row, dtype)) return s;
    if (int s = check_rows(fn, "out", out, out_stride, row, dtype)) return s;
    if (out == x && out_stride != x_stride && N > 1)
        return fail(BITNET_E_SHAPE, "%s: out is x with another stride", fn);
    if (!positions) return fail(BITNET_E_NULL, "%s: positions is required", fn);
    if (!aligned(positions, 4))
        return fail(BITNET_E_ALIGN, "%s: positions must be 4-byte aligned", fn);
    const bitnet::RotaryArgs r{plan->turns, plan->magnitude, inverse ? -1.0 : 1.0, (int)plan->rot,
                               plan->interleaved != 0};
    hipError_t e = bitnet::launch_rotary(r, x, x_stride, out, out_stride, dtype == BITNET_BF16, N,
                                         (int)n_heads, (int)head_dim, positions,
                                         static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(fn, e);
    return ok();
}

BITNET_API int bitnet_rotary_kv4_append(const bitnet_kv4_batch *batch,
                                        const bitnet_rotary_plan *plan, const void *q,
                                        int64_t q_stride, void *q_out, int64_t out_stride,
                                        int64_t n_heads, const void *k, int64_t k_stride,
                                        const void *v, int64_t v_stride, int dtype, int64_t N,
                                        const int32_t *offset, void *stream) {
    const char *fn = "bitnet_rotary_kv4_append";
    if (int s = check_kv4(fn, batch, dtype, N)) return s;
    if (int s = check_heads(fn, n_heads, batch->n_kv_heads)) return s;
    if (int s = check_plan(fn, plan, batch->head_dim)) return s;
    if (N == 0 || batch->n_seqs == 0) return ok();
    if (int s = check_turns(fn, plan)) return s;
    const int64_t row = batch->n_kv_heads * batch->head_dim, q_row = n_heads * batch->head_dim;
    if (int s = check_rows(fn, "q", q, q_stride, q_row, dtype)) return s;
    if (int s = check_rows(fn, "q_out", q_out, out_stride, q_row, dtype)) return s;
    if (q_out == q && out_stride != q_stride && N > 1)
        return fail(BITNET_E_SHAPE, "%s: q_out is q with another stride", fn);
    if (int s = check_rows(fn, "k", k, k_stride, row, dtype)) return s;
    if (int s = check_rows(fn, "v", v, v_stride, row, dtype)) return s;
    if (!aligned(offset, 4)) return fail(BITNET_E_ALIGN, "%s: offset must be 4-byte aligned", fn);
    const bitnet::RotaryArgs r{plan->turns, plan->magnitude, 1.0, (int)plan->rot,
                               plan->interleaved != 0};
    hipError_t e = bitnet::launch_rotary_append(
        r, kv4_args(batch), q, q_stride, q_out, out_stride, (int)n_heads, k, k_stride, v, v_stride,
        offset, dtype == BITNET_BF16, N, (int)batch->head_dim, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(fn, e);
    return ok();
}

static int check_w4(const char *fn, const bitnet_w4_matrix *m) {
    if (!m) return fail(BITNET_E_NULL, "%s: mat is NULL", fn);
    if (m->M < 0 || m->M > BITNET_W4_MAX_ROWS)
        return fail(BITNET_E_SHAPE, "%s: M=%lld outside [0, %d]", fn, (long long)m->M,
                    BITNET_W4_MAX_ROWS);
    if (int s = check_k(fn, m->K)) return s;
    const int64_t group = m->group & ~(int64_t)BITNET_W4_BY_GROUP;
    if (group != 32 && group != 64 && group != 128)
        return fail(BITNET_E_SHAPE, "%s: group=%lld must be 32, 64 or 128", fn, (long long)m->group);
    if (m->M == 0) return BITNET_OK;
    if (!m->codes || !m->steps) return fail(BITNET_E_NULL, "%s: codes and steps are required", fn);
    if (!aligned(m->codes, 16) || !aligned(m->steps, 16))
        return fail(BITNET_E_ALIGN, "%s: codes and steps must be 16-byte aligned", fn);
    return BITNET_OK;
}
static bitnet::W4Args w4_args(const bitnet_w4_matrix *m) {
    const int64_t group = m->group & ~(int64_t)BITNET_W4_BY_GROUP;
    return bitnet::W4Args{static_cast<uint8_t *>(m->codes), static_cast<uint16_t *>(m->steps),
                          (int)m->M, (int)m->K, (int)(128 / group), m->group != group};
}
static int pack_w4(const char *fn, const void *w, int form, const void *given,
                   const bitnet_w4_matrix *m, void *stream) {
    hipError_t e = bitnet::launch_w4_pack(w, form, static_cast<const uint16_t *>(given), w4_args(m),
                                          static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(fn, e);
    return ok();
}

BITNET_API int bitnet_pack_w4(const void *w, int dtype, const bitnet_w4_matrix *mat, void *stream) {
    const char *fn = "bitnet_pack_w4";
    if (dtype != BITNET_F32 && dtype != BITNET_BF16)
        return fail(BITNET_E_DTYPE, "%s: unknown dtype %d", fn, dtype);
    if (int s = check_w4(fn, mat)) return s;
    if (mat->M == 0) return ok();
    if (!w) return fail(BITNET_E_NULL, "%s: w is required", fn);
    if (!aligned(w, 16)) return fail(BITNET_E_ALIGN, "%s: w must be 16-byte aligned", fn);
    return pack_w4(fn, w, dtype == BITNET_BF16, nullptr, mat, stream);
}

BITNET_API int bitnet_pack_w4_codes(const int8_t *w, const void *given, const bitnet_w4_matrix *mat,
                                    void *stream) {
    const char *fn = "bitnet_pack_w4_codes";
    if (int s = check_w4(fn, mat)) return s;
    if (mat->M == 0) return ok();
    if (!w || !given) return fail(BITNET_E_NULL, "%s: w and given are required", fn);
    if (!aligned(w, 8) || !aligned(given, 2))
        return fail(BITNET_E_ALIGN, "%s: w must be 8-byte and given 2-byte aligned", fn);
    return pack_w4(fn, w, 2, given, mat, stream);
}

BITNET_API int bitnet_w4_rows(const bitnet_w4_matrix *mat, const int32_t *ids, int64_t n, void *out,
                              int dtype, void *stream) {
    const char *fn = "bitnet_w4_rows";
    if (dtype != BITNET_F32 && dtype != BITNET_BF16)
        return fail(BITNET_E_DTYPE, "%s: unknown dtype %d", fn, dtype);
    if (n < 0 || n > BITNET_GEMM_MAX_N)
        return fail(BITNET_E_SHAPE, "%s: n=%lld outside [0, %d]", fn, (long long)n,
                    BITNET_GEMM_MAX_N);
    if (int s = check_w4(fn, mat)) return s;
    if (n == 0) return ok();
    if (!out) return fail(BITNET_E_NULL, "%s: out is required", fn);
    if (!aligned(out, 16)) return fail(BITNET_E_ALIGN, "%s: out must be 16-byte aligned", fn);
    if (!aligned(ids, 4)) return fail(BITNET_E_ALIGN, "%s: ids must be 4-byte aligned", fn);
    hipError_t e = bitnet::launch_w4_rows(w4_args(mat), ids, n, out, dtype == BITNET_BF16,
                                          static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(fn, e);
    return ok();
}

BITNET_API int64_t bitnet_linear_w4_workspace(int64_t N, int64_t M, int64_t K) {
    const char *fn = "bitnet_linear_w4_workspace";
    if (check_k(fn, K)) return -1;
    if (N < 0 || N > BITNET_GEMM_MAX_N || M < 0 || M > BITNET_W4_MAX_ROWS) {
        fail(BITNET_E_SHAPE, "%s: sizes out of range", fn);
        return -1;
    }
    g_last_error.clear();
    if (N == 0 || M == 0) return 0;
    const int64_t shares = bitnet::w4_plan(N, M, K).shares;
    return shares > 1 ? shares * N * M * 4 : 0;
}

BITNET_API int bitnet_linear_w4(const void *x, int dtype, int64_t N, const bitnet_w4_matrix *mat,
                                float *y, void *workspace, int64_t workspace_bytes, void *stream) {
    const char *fn = "bitnet_linear_w4";
    if (dtype != BITNET_F32 && dtype != BITNET_BF16)
        return fail(BITNET_E_DTYPE, "%s: unknown dtype %d", fn, dtype);
    if (N < 0 || N > BITNET_GEMM_MAX_N)
        return fail(BITNET_E_SHAPE, "%s: N=%lld outside [0, %d]", fn, (long long)N,
                    BITNET_GEMM_MAX_N);
    if (int s = check_w4(fn, mat)) return s;
    if (N == 0 || mat->M == 0) return ok();
    if (!x || !y) return fail(BITNET_E_NULL, "%s: x and y are required", fn);
    if (!aligned(x, 16) || !aligned(y, 4) || !aligned(workspace, 16))
        return fail(BITNET_E_ALIGN, "%s: x and workspace must be 16-byte and y 4-byte aligned", fn);
    const bitnet::W4Plan p = bitnet::w4_plan(N, mat->M, mat->K);
    const int64_t need = p.shares > 1 ? p.shares * N * mat->M * 4 : 0;
    if (need > 0 && !workspace)
        return fail(BITNET_E_NULL, "%s: a workspace of %lld bytes is required", fn, (long long)need);
    if (workspace_bytes < need)
        return fail(BITNET_E_SHAPE, "%s: the workspace has %lld bytes, %lld are required", fn,
                    (long long)workspace_bytes, (long long)need);
    hipError_t e = bitnet::launch_w4_linear(w4_args(mat), x, dtype == BITNET_BF16, N, y,
                                            static_cast<float *>(workspace), p,
                                            static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(fn, e);
    return ok();
}

#ifdef BITNET_STAMPS
// Instrumented build only (include/bitnet_i2s_stamps.h).
namespace bitnet {
int stamps_reset(int rewind, hipStream_t st);
int stamps_read(unsigned long long *out, int max_launches);
}  // namespace bitnet

BITNET_API int bitnet_stamps_reset(int rewind, void *stream) {
    if (bitnet::stamps_reset(rewind, static_cast<hipStream_t>(stream)) != 0)
        return fail(BITNET_E_HIP, "bitnet_stamps_reset: no stamp slots on this device");
    return ok();
}

BITNET_API int bitnet_stamps_read(uint64_t *out, int max_launches) {
    if (!out && max_launches > 0) return -1;
    return bitnet::stamps_read(reinterpret_cast<unsigned long long *>(out), max_launches);
}
#endif
