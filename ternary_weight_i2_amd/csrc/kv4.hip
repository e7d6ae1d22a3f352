// kv4.hip -- the 4-bit key/value cache: quantising keys and values as they are
// written, and reading them back (kv4.h: the quantiser and the layout).
//
// Eight lanes hold a group of 64 channels, eight channels each: its smallest
// and largest value come from three DPP moves, every lane quantises its own
// eight and stores them.  Both kernels are bound by HBM for prompts (5 or 3
// bytes a value with fp32 or bf16 rows) and by latency for single tokens.
#include "kv4.h"

namespace bitnet {

namespace {

constexpr int kKvThreads = 256;

__device__ __forceinline__ float min8(float v) {   // over 8 aligned lanes
    v = fminf(v, dpp_f32<kDppXor1>(v));
    v = fminf(v, dpp_f32<kDppXor2>(v));
    return fminf(v, dpp_f32<kDppHalfMirror>(v));
}
__device__ __forceinline__ float max8(float v) {
    v = fmaxf(v, dpp_f32<kDppXor1>(v));
    v = fmaxf(v, dpp_f32<kDppXor2>(v));
    return fmaxf(v, dpp_f32<kDppHalfMirror>(v));
}

// The group's pair (step in the low half) and this lane's eight codes.
__device__ __forceinline__ uint32_t quantise8(float (&x)[8], uint32_t *pair) {
#pragma clang fp contract(off)
    float lo = kKv4Max, hi = -kKv4Max;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        x[e] = fminf(fmaxf(x[e], -kKv4Max), kKv4Max);   // a NaN becomes -kKv4Max
        lo = fminf(lo, x[e]);
        hi = fmaxf(hi, x[e]);
    }
    lo = min8(lo);
    hi = max8(hi);
    const _Float16 mid16 = (_Float16)(lo + (hi - lo) * (8.0f / 15.0f));
    const float mid = (float)mid16;
    const _Float16 step16 = (_Float16)fmaxf((hi - mid) * (1.0f / 7.0f), (mid - lo) * 0.125f);
    const float step = (float)step16;
    const float inv = step > 0.0f ? 1.0f / step : 0.0f;
    uint32_t codes = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float t = (x[e] - mid) * inv;
        const float c = fminf(fmaxf(rintf(t + 8.0f), 0.0f), 15.0f);
        codes |= (uint32_t)c << (4 * e);
    }
    *pair = (uint32_t)__builtin_bit_cast(uint16_t, step16) |
            (uint32_t)__builtin_bit_cast(uint16_t, mid16) << 16;
    return codes;
}

template <int D, bool BF16>
__global__ __launch_bounds__(kKvThreads) void kv4_append_kernel(
    const Kv4Args c, const void *k, const void *v, int64_t k_stride, int64_t v_stride, int64_t N) {
    using L = Kv4Page<D>;
    // one lane: eight channels of a (token, head, key or value) row
    const int64_t i = (int64_t)blockIdx.x * kKvThreads + threadIdx.x;
    const int p = (int)(i % (D / 8));
    int64_t r = i / (D / 8);
    const int is_v = (int)(r & 1);
    r >>= 1;
    const int head = (int)(r % c.kv_heads);
    const int64_t token = r / c.kv_heads;
    if (token >= N) return;   // whole groups of eight lanes leave together
    const Kv4Place at = place_of(c, token);
    if (at.rec < 0) return;
    float x[8];
    load8<BF16>(is_v ? v : k, token * (is_v ? v_stride : k_stride) + head * D + 8 * p, x);
    uint32_t pair;
    const uint32_t codes = quantise8(x, &pair);
    uint8_t *rec = c.cache + (at.rec + head) * (int64_t)L::kBytes;
    const int g = p >> 3, t = at.in_page;
    if (!is_v) {
        const int dw = t * (D / 8) + (p & 3) * L::kSteps + (p >> 2);
        reinterpret_cast<uint32_t *>(rec)[dw] = codes;
        if ((p & 7) == 0)
            reinterpret_cast<uint32_t *>(rec + L::kKeyPairs)[t * L::kGroups + g] = pair;
    } else {
        uint16_t *w = reinterpret_cast<uint16_t *>(rec + L::kValues);
        const int lane = 2 * (p & 7), blk = t >> 2;
        w[((blk * 16 + lane) * L::kGroups + g) * 4 + (t & 3)] = (uint16_t)codes;
        w[((blk * 16 + lane + 1) * L::kGroups + g) * 4 + (t & 3)] = (uint16_t)(codes >> 16);
        if ((p & 7) == 0) {
            uint16_t *m = reinterpret_cast<uint16_t *>(rec + L::kValuePairs);
            m[(blk * L::kGroups + g) * 8 + (t & 3)] = (uint16_t)pair;
            m[(blk * L::kGroups + g) * 8 + 4 + (t & 3)] = (uint16_t)(pair >> 16);
        }
    }
}

template <int D, bool BF16>
__global__ __launch_bounds__(kKvThreads) void kv4_read_kernel(const Kv4Args c, void *k, void *v,
                                                              int64_t N) {
#pragma clang fp contract(off)
    using L = Kv4Page<D>;
    const int64_t i = (int64_t)blockIdx.x * kKvThreads + threadIdx.x;
    const int p = (int)(i % (D / 8));
    int64_t r = i / (D / 8);
    const int is_v = (int)(r & 1);
    r >>= 1;
    const int head = (int)(r % c.kv_heads);
    const int64_t token = r / c.kv_heads;
    void *out = is_v ? v : k;
    if (token >= N || !out || !row_in_call(c, token)) return;
    const Kv4Place at = place_of(c, token);
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = 0.0f;
    if (at.rec >= 0) {
        const uint8_t *rec = c.cache + (at.rec + head) * (int64_t)L::kBytes;
        const int g = p >> 3, t = at.in_page;
        uint32_t codes, pair;
        if (!is_v) {
            codes = reinterpret_cast<const uint32_t *>(
                rec)[t * (D / 8) + (p & 3) * L::kSteps + (p >> 2)];
            pair = reinterpret_cast<const uint32_t *>(rec + L::kKeyPairs)[t * L::kGroups + g];
        } else {
            const uint16_t *w = reinterpret_cast<const uint16_t *>(rec + L::kValues);
            const uint16_t *m = reinterpret_cast<const uint16_t *>(rec + L::kValuePairs);
            const int lane = 2 * (p & 7), blk = t >> 2;
            codes = w[((blk * 16 + lane) * L::kGroups + g) * 4 + (t & 3)] |
                    (uint32_t)w[((blk * 16 + lane + 1) * L::kGroups + g) * 4 + (t & 3)] << 16;
            pair = m[(blk * L::kGroups + g) * 8 + (t & 3)] |
                   (uint32_t)m[(blk * L::kGroups + g) * 8 + 4 + (t & 3)] << 16;
        }
        const float step = (float)__builtin_bit_cast(_Float16, (uint16_t)pair);
        const float mid = (float)__builtin_bit_cast(_Float16, (uint16_t)(pair >> 16));
#pragma unroll
        for (int e = 0; e < 8; ++e)
            x[e] = mid + step * (float)((int)((codes >> (4 * e)) & 15u) - 8);
    }
    const int64_t o = (token * c.kv_heads + head) * D + 8 * p;
    if constexpr (BF16) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = bf16_bits(x[2 * e]) | bf16_bits(x[2 * e + 1]) << 16;
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out) + o) =
            make_uint4(w[0], w[1], w[2], w[3]);
    } else {
        float4 *f = reinterpret_cast<float4 *>(static_cast<float *>(out) + o);
        f[0] = make_float4(x[0], x[1], x[2], x[3]);
        f[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
}

}  // namespace

hipError_t launch_kv4_append(const Kv4Args &c, const void *k, const void *v, int bf16,
                             int64_t k_stride, int64_t v_stride, int64_t N, int dim,
                             hipStream_t st) {
    const int64_t lanes = N * c.kv_heads * 2 * (dim / 8);
    const dim3 g((unsigned)((lanes + kKvThreads - 1) / kKvThreads)), t(kKvThreads);
#define KV4_APPEND(D, B) \
    hipLaunchKernelGGL((kv4_append_kernel<D, B>), g, t, 0, st, c, k, v, k_stride, v_stride, N)
    if (dim == 64) { if (bf16) KV4_APPEND(64, true); else KV4_APPEND(64, false); }
    else if (dim == 128) { if (bf16) KV4_APPEND(128, true); else KV4_APPEND(128, false); }
    else { if (bf16) KV4_APPEND(256, true); else KV4_APPEND(256, false); }
#undef KV4_APPEND
    return hipGetLastError();
}

hipError_t launch_kv4_read(const Kv4Args &c, void *k, void *v, int bf16, int64_t N, int dim,
                           hipStream_t st) {
    const int64_t lanes = N * c.kv_heads * 2 * (dim / 8);
    const dim3 g((unsigned)((lanes + kKvThreads - 1) / kKvThreads)), t(kKvThreads);
#define KV4_READ(D, B) hipLaunchKernelGGL((kv4_read_kernel<D, B>), g, t, 0, st, c, k, v, N)
    if (dim == 64) { if (bf16) KV4_READ(64, true); else KV4_READ(64, false); }
    else if (dim == 128) { if (bf16) KV4_READ(128, true); else KV4_READ(128, false); }
    else { if (bf16) KV4_READ(256, true); else KV4_READ(256, false); }
#undef KV4_READ
    return hipGetLastError();
}

}  // namespace bitnet
