// kv4.hip -- the 4-bit key/value cache: quantising keys and values as they are
// written, and reading them back (kv4.h: the quantiser and the layout).
//
// A workgroup takes four positions of one sequence that lie side by side in a page
// (a block of the value codes), all heads, keys and values.  Eight lanes hold a
// group of 64 channels, eight channels each, of all four tokens: a group's ends come
// from three DPP moves, and a lane's value codes are two stores of 8 bytes, 16 side
// by side for a group.  Both kernels are bound by HBM for prompts (4.56 or 2.56
// bytes a value with fp32 or bf16 rows): 6800 rows of 8 heads of 128, bf16, 35.6 MB
// each way, are written in 12.8 us and read back in 10.1 (2.8 and 3.5 TB/s; in a graph
// 11.0 and 9.3, where a copy that moves as much takes 6.1); 20000 fp32 rows of 5 heads
// read in 24 us (119 MB, 4.9 TB/s).  Single tokens are bound by latency, the loads of
// the lengths, the table and the rows: 64 of them 4.0 and 3.2 us.
#include "kv4.h"

namespace bitnet {

namespace {

constexpr int kKvThreads = 256;

template <int D, bool BF16>
__global__ __launch_bounds__(kKvThreads) void kv4_append_kernel(
    const Kv4Args c, const void *k, const void *v, int64_t k_stride, int64_t v_stride, int64_t N) {
    using L = Kv4Page<D>;
    const Block4 at = find_block(c, N);
    if (!at.rows) return;   // the whole workgroup
    const int lanes = c.kv_heads * 2 * (D / 8), t0 = at.in_page;
    for (int i = threadIdx.x; i < lanes; i += blockDim.x) {   // whole groups of eight lanes
        const int p = i % (D / 8), head = i / (D / 8) >> 1;
        const bool is_v = i / (D / 8) & 1;
        const void *src = is_v ? v : k;
        const int64_t stride = is_v ? v_stride : k_stride;
        float x[4][8];
#pragma unroll
        for (int t = 0; t < 4; ++t)
            if (at.rows >> t & 1)
                load8<BF16>(src, (at.row + t) * stride + head * D + 8 * p, x[t]);
        uint32_t codes[4], pair[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) codes[t] = quantise8(x[t], &pair[t]);
        if (!at.cached(c)) return;   // the whole workgroup; the rows are on their way by now
        uint8_t *rec = c.cache + ((int64_t)at.page * c.kv_heads + head) * L::kBytes;
        store_block4<D>(rec, is_v, t0, p, at.rows, codes, pair);
    }
}

template <int D, bool BF16>
__global__ __launch_bounds__(kKvThreads) void kv4_read_kernel(const Kv4Args c, void *k, void *v,
                                                              int64_t N) {
#pragma clang fp contract(off)
    using L = Kv4Page<D>;
    const Block4 at = find_block(c, N);
    if (!at.rows) return;   // the whole workgroup
    const int lanes = c.kv_heads * 2 * (D / 8), t0 = at.in_page;
    for (int i = threadIdx.x; i < lanes; i += blockDim.x) {
        const int p = i % (D / 8), g = p >> 3, head = i / (D / 8) >> 1;
        const bool is_v = i / (D / 8) & 1;
        void *out = is_v ? v : k;
        if (!out) continue;
        uint32_t codes[4] = {0, 0, 0, 0}, pair[4] = {0, 0, 0, 0};   // zeros where there is no page
        if (at.cached(c)) {
            const uint8_t *rec = c.cache + ((int64_t)at.page * c.kv_heads + head) * L::kBytes;
            if (!is_v) {
                const uint32_t *w = reinterpret_cast<const uint32_t *>(rec) + t0 * (D / 8) +
                                    (p & 3) * L::kSteps + (p >> 2);
                const uint32_t *m =
                    reinterpret_cast<const uint32_t *>(rec + L::kKeyPairs) + t0 * L::kGroups + g;
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    codes[t] = w[t * (D / 8)];
                    pair[t] = m[t * L::kGroups];
                }
            } else {
                const uint16_t *w = reinterpret_cast<const uint16_t *>(rec + L::kValues) +
                                    ((t0 >> 2) * 16 + 2 * (p & 7)) * L::kGroups * 4 + g * 4;
                const uint2 a = *reinterpret_cast<const uint2 *>(w);
                const uint2 b = *reinterpret_cast<const uint2 *>(w + 4 * L::kGroups);
                const uint4 m = *reinterpret_cast<const uint4 *>(
                    rec + L::kValuePairs + ((t0 >> 2) * L::kGroups + g) * 16);
                codes[0] = (a.x & 0xffffu) | b.x << 16;
                codes[1] = a.x >> 16 | (b.x & 0xffff0000u);
                codes[2] = (a.y & 0xffffu) | b.y << 16;
                codes[3] = a.y >> 16 | (b.y & 0xffff0000u);
                pair[0] = (m.x & 0xffffu) | m.z << 16;
                pair[1] = m.x >> 16 | (m.z & 0xffff0000u);
                pair[2] = (m.y & 0xffffu) | m.w << 16;
                pair[3] = m.y >> 16 | (m.w & 0xffff0000u);
            }
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            if (!(at.rows >> t & 1)) continue;
            const float step = (float)__builtin_bit_cast(_Float16, (uint16_t)pair[t]);
            const float mid = (float)__builtin_bit_cast(_Float16, (uint16_t)(pair[t] >> 16));
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                x[e] = mid + step * (float)((int)((codes[t] >> (4 * e)) & 15u) - 8);
            const int64_t o = ((int64_t)(at.row + t) * c.kv_heads + head) * D + 8 * p;
            if constexpr (BF16) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    w[e] = bf16_bits(x[2 * e]) | bf16_bits(x[2 * e + 1]) << 16;
                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out) + o) =
                    make_uint4(w[0], w[1], w[2], w[3]);
            } else {
                float4 *f = reinterpret_cast<float4 *>(static_cast<float *>(out) + o);
                f[0] = make_float4(x[0], x[1], x[2], x[3]);
                f[1] = make_float4(x[4], x[5], x[6], x[7]);
            }
        }
    }
}

// A sequence of n rows touches at most n / 4 + 2 blocks.
dim3 block_grid(const Kv4Args &c, int64_t N) { return dim3((unsigned)(N / 4 + 2 * c.n_seqs)); }
dim3 block_threads(const Kv4Args &c, int dim) {
    const int lanes = c.kv_heads * 2 * (dim / 8);
    return dim3(lanes < kKvThreads ? (lanes + 63) / 64 * 64 : kKvThreads);
}

}  // namespace

hipError_t launch_kv4_append(const Kv4Args &c, const void *k, const void *v, int bf16,
                             int64_t k_stride, int64_t v_stride, int64_t N, int dim,
                             hipStream_t st) {
    const dim3 g = block_grid(c, N), t = block_threads(c, dim);
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
    const dim3 g = block_grid(c, N), t = block_threads(c, dim);
#define KV4_READ(D, B) hipLaunchKernelGGL((kv4_read_kernel<D, B>), g, t, 0, st, c, k, v, N)
    if (dim == 64) { if (bf16) KV4_READ(64, true); else KV4_READ(64, false); }
    else if (dim == 128) { if (bf16) KV4_READ(128, true); else KV4_READ(128, false); }
    else { if (bf16) KV4_READ(256, true); else KV4_READ(256, false); }
#undef KV4_READ
    return hipGetLastError();
}

}  // namespace bitnet
