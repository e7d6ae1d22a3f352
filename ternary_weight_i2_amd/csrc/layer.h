// layer.h -- device helpers and launcher declarations of what stands between a
// layer's matmuls: the block boundary, the 4-bit cache and its attention
// (library-internal; not installed).
#pragma once

#include "attn_plan.h"
#include "common.h"
#include "w4_plan.h"

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
// One value of a bf16 or fp32 row, read as fp32 and stored rounded to nearest even.
template <bool BF16>
__device__ __forceinline__ float load1(const void *p, int64_t i) {
    if constexpr (BF16)
        return __uint_as_float((uint32_t) static_cast<const uint16_t *>(p)[i] << 16);
    else
        return static_cast<const float *>(p)[i];
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

// Stores eight values, bf16 rounded to nearest even.
template <bool BF16>
__device__ __forceinline__ void store8_values(void *p, int64_t i, const float (&x)[8]) {
    if constexpr (BF16) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = bf16_bits(x[2 * e]) | bf16_bits(x[2 * e + 1]) << 16;
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + i) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
        float4 *f = reinterpret_cast<float4 *>(static_cast<float *>(p) + i);
        f[0] = make_float4(x[0], x[1], x[2], x[3]);
        f[1] = make_float4(x[4], x[5], x[6], x[7]);
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
// Rotary positions (rotary.hip): turns per position of each pair of channels, as 64-bit
// fractions of one.
struct RotaryArgs {
    const int64_t *turns;
    double magnitude, sign;   // sign: -1 turns back
    int rot, interleaved;
};
hipError_t launch_rotary(const RotaryArgs &r, const void *x, int64_t x_stride, void *out,
                         int64_t out_stride, int bf16, int64_t N, int heads, int dim,
                         const int32_t *positions, hipStream_t st);
hipError_t launch_rotary_append(const RotaryArgs &r, const Kv4Args &c, const void *q,
                                int64_t q_stride, void *q_out, int64_t out_stride, int heads,
                                const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                                const int32_t *offset, int bf16, int64_t N, int dim,
                                hipStream_t st);
// A matrix of 4-bit weights (w4.hip has its layout); groups: steps of a row's 128 channels,
// by_group: these lie group by group, not row by row.
struct W4Args {
    uint8_t *codes;
    uint16_t *steps;
    int M, K, groups, by_group;
};
hipError_t launch_w4_pack(const void *w, int form, const uint16_t *given, const W4Args &to, hipStream_t st);
hipError_t launch_w4_rows(const W4Args &w, const int32_t *ids, int64_t n, void *out, int bf16,
                          hipStream_t st);
hipError_t launch_w4_linear(const W4Args &w, const void *x, int bf16, int64_t N, float *y,
                            float *part, const W4Plan &plan, hipStream_t st);
// The attention weights of a call's rows, summed by cached token (kv4_weigh.hip).
struct WeighArgs {
    Kv4Args c;
    const void *q;
    const float *old;
    float *out;
    float2 *part;          // per split and row: maximum and sum
    uint4 *kept;           // many rows: the queries as operands
    float *sums;           // many rows, few pages: the parts' sums
    int64_t q_stride, N;
    float scale_log2, decay;
    int heads, window, sinks, splits;   // splits: WeighPlan
};
hipError_t launch_kv4_weigh(const WeighArgs &a, const WeighPlan &plan, int bf16, int dim,
                            hipStream_t st);
// The tokens of the largest weight, moved to other pages (kv4_evict.hip).
struct EvictArgs {
    uint8_t *cache;
    float *weights;
    const int32_t *table, *kv_len, *new_table;
    int32_t *new_len, *index;
    int *counts;           // several workgroups to a choice: EvictPlan
    int2 *search, *slices;
    int64_t n_pages, max_pages, new_pages, n_seqs;
    int kv_heads, keep, sinks, recent;
};
hipError_t launch_kv4_evict(const EvictArgs &a, const EvictPlan &plan, int dim, hipStream_t st);
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
