// layer.h -- device helpers and launcher declarations of what stands between a
// layer's matmuls: the block boundary, the 4-bit cache and its attention
// (library-internal; not installed).
#pragma once

#include "attn_plan.h"
#include "common.h"

namespace bitnet {

// Wave-wide sum of doubles, returned to every lane, always added in the same
// order (exact for integer multiples below 2^53).
__device__ __forceinline__ double wave_sum_f64(double v) {
    uint64_t b;
    __builtin_memcpy(&b, &v, 8);
    auto add = [&](uint64_t o) {
        double x, y;
        __builtin_memcpy(&x, &b, 8);
        __builtin_memcpy(&y, &o, 8);
        x += y;
        __builtin_memcpy(&b, &x, 8);
    };
    add(dpp_u64<kDppXor1>(b));
    add(dpp_u64<kDppXor2>(b));
    add(dpp_u64<kDppHalfMirror>(b));
    add(dpp_u64<kDppMirror>(b));
    add(dpp_rows_u64<kDppRowBcast15, 0xA>(b));   // the rows a move skips add +0
    add(dpp_rows_u64<kDppRowBcast31, 0xC>(b));
    b = readlane63_u64(b);
    double r;
    __builtin_memcpy(&r, &b, 8);
    return r;
}

// The bf16 nearest to v, half to even (finite v).
__device__ __forceinline__ uint32_t bf16_bits(float v) {
    const uint32_t u = __float_as_uint(v);
    return (u + 0x7fffu + ((u >> 16) & 1u)) >> 16;
}
// Eight consecutive values of a bf16 or fp32 row, as fp32.
template <bool BF16>
__device__ __forceinline__ void load8(const void *p, int64_t i, float (&x)[8]) {
    if constexpr (BF16) {
        const uint4 r = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + i);
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[2 * e] = __uint_as_float(w[e] << 16);
            x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
        }
    } else {
        const float4 a = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
        const float4 b = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i + 4);
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
}

// ---- launchers (each returns the hipError_t of its launch) ---------------
// The boundary between two blocks: norm, gate, scale, residual, norm, tokens;
// one workgroup per token (F a multiple of 128, at most 32768).
struct BlockNormArgs {
    const void *b;
    const float *post_gamma, *gate, *gamma;
    const void *res;
    void *h, *v;
    int8_t *xq;
    float *xs;
    int32_t *xsum;
    int64_t gate_stride;   // 0: one gate row for every token
    float scale, eps;
    int F, post;
};
hipError_t launch_block_norm(const BlockNormArgs &a, int64_t N, int b_bf16, int s_bf16,
                             hipStream_t st);

// The 4-bit key/value cache (kv4.h has its layout) and the sequences of a call.
struct Kv4Args {
    uint8_t *cache;
    const int32_t *table, *kv_len, *q_start;
    int64_t n_pages, max_pages, n_seqs;
    int kv_heads;
};
hipError_t launch_kv4_append(const Kv4Args &c, const void *k, const void *v, int bf16,
                             int64_t k_stride, int64_t v_stride, int64_t N, int dim,
                             hipStream_t st);
hipError_t launch_kv4_read(const Kv4Args &c, void *k, void *v, int bf16, int64_t N, int dim,
                           hipStream_t st);
struct Attn4Args {
    Kv4Args c;
    const void *q;
    void *out;
    float *part;           // per split, row: dim accumulators, then maximum and sum
    int64_t q_stride, N;
    float scale_log2;      // softmax scale times log2(e)
    int heads, window, sinks, splits;   // splits and `tiles`: Attn4Plan
    uint32_t tiles;
};
hipError_t launch_attn4(const Attn4Args &a, const Attn4Plan &plan, int bf16, int dim,
                        hipStream_t st);

}  // namespace bitnet
