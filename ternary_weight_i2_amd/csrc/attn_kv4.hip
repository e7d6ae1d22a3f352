// attn_kv4.hip -- causal attention over the 4-bit cache (kv4.h: its layout),
// with an optional sliding window and a few first tokens that stay visible.
//
//   out[row] = sum_t p_t v_t / sum_t p_t,   p_t = 2^(x_t - max x),
//   x_t = log2(e) * scale * q . k_t
// in one pass over the pages with a running maximum.  The queries of all heads
// that share a kv head are rows of one problem: row r of a sequence is token
// r / G, head r % G of the group.
//
// Both products run on the fp16 16x16x32 matrix instruction with the codes as
// they are: code - 8 is a small integer, exact in fp16, and one packed
// operation away from the stored nibble.  For a group of 64 channels
//   q . k_t = sum_g step_tg (q_g . code_tg) + mid_tg sum(q_g)
//   sum_t p_t v_t = sum_t (p_t step_tg) code_tg + sum_t p_t mid_tg
// so the pairs enter in fp32 after the first product and through p * step in
// front of the second.  q is scaled by a power of two per row, p * step by one
// per wave (from the largest step met so far, tracked like the maximum), so
// neither leaves fp16's normal range; bf16 calls round both once to fp16 (8 and
// 11 bits: finer than the output), fp32 calls carry them as two fp16 terms (22
// bits).  Sums, maxima and accumulators are fp32.
//
// The first product is taken transposed (tokens x rows), which leaves a lane
// with 16 tokens of one row: that is exactly the fragment that the second
// product (channels x rows) takes, so p never crosses lanes, and the running
// maximum, the sum and the accumulators of a row all live in the same lanes.
#include "kv4.h"

namespace bitnet {

namespace {

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));

constexpr int kRows = 16;          // rows of a tile
constexpr int kWaves = 4;          // waves of a workgroup; each takes every fourth page
constexpr float kNoMax = -3.0e38f; // a running maximum before the first visible token

__device__ __forceinline__ h2 as_h2(uint32_t w) { return __builtin_bit_cast(h2, w); }
__device__ __forceinline__ h8 join(h2 a, h2 b, h2 c, h2 d) {
    return h8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Eight nibbles of a word as code - 8, in the order 0 4, 1 5, 2 6, 3 7.  A
// nibble in the low mantissa bits of 1024 = 0x6400 makes 1024 + code (or 1024 +
// 16 code one place up); both results are exact.
__device__ __forceinline__ void codes8(uint32_t w, h2 (&c)[4]) {
    const uint32_t one = 0x64006400u;
    const h2 s = {(_Float16)0.0625f, (_Float16)0.0625f};
    const uint32_t w8 = w >> 8;
    c[0] = as_h2((w & 0x000f000fu) | one) - (_Float16)1032.0f;
    c[1] = as_h2((w & 0x00f000f0u) | one) * s - (_Float16)72.0f;
    c[2] = as_h2((w8 & 0x000f000fu) | one) - (_Float16)1032.0f;
    c[3] = as_h2((w8 & 0x00f000f0u) | one) * s - (_Float16)72.0f;
}

// Over the four lanes that hold a row (l, l ^ 16, l ^ 32, l ^ 48).
__device__ __forceinline__ float quad_max(float v) {
    v = fmaxf(v, __shfl_xor(v, 16));
    return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float quad_sum(float v) {
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

// The tile (16 rows of one sequence) that a workgroup works on, and the pages
// its rows see: the first `sink_pages`, then from `first` to `last`.
struct Tile {
    int64_t seq, token0, rows, row0, held;   // token0: the sequence's first query token
    int64_t pos0;                            // position of row 0's token
    int64_t first, sink_pages, pages;
};

__device__ __forceinline__ Tile find_tile(const Attn4Args &a, int64_t x, int G) {
    Tile t;
    // the largest b with q_start[b] * G / 16 + b <= x: a sequence has at least
    // as many tiles to itself as its rows need
    int64_t lo = 0, hi = a.c.n_seqs - 1;
    while (lo < hi) {
        const int64_t m = (lo + hi + 1) >> 1;
        if ((int64_t)a.c.q_start[m] * G / kRows + m <= x) lo = m;
        else hi = m - 1;
    }
    t.seq = lo;
    const int64_t begin = a.c.q_start[lo], end = a.c.q_start[lo + 1];
    t.token0 = begin;
    t.rows = end > begin && begin >= 0 && end <= a.N ? (end - begin) * G : 0;
    t.row0 = (x - (begin * G / kRows + lo)) * kRows;
    if (t.row0 < 0) t.rows = 0;
    t.held = held_tokens(a.c, lo);
    t.pos0 = t.held - (end - begin);
    t.pages = t.first = t.sink_pages = 0;
    if (t.row0 >= t.rows) return t;
    const int64_t last_row = min(t.row0 + kRows, t.rows) - 1;
    const int64_t pos_a = t.pos0 + t.row0 / G, pos_b = t.pos0 + last_row / G;
    if (pos_b < 0) return t;
    t.first = a.window > 0 && pos_a >= a.window ? (pos_a - a.window + 1) / kPage : 0;
    t.sink_pages = min((a.sinks + kPage - 1) / kPage, t.first);
    t.pages = t.sink_pages + pos_b / kPage - t.first + 1;
    return t;
}

template <int D>
struct RawPage {   // a page's codes as one lane loads them, and its share of the pairs
    uint32_t k[4][D / 32];
    uint32_t v[4][D / 32];
    uint32_t m[D / 32];
};

template <int N>
__device__ __forceinline__ void load_words(const uint8_t *p, uint32_t (&w)[N]) {
    static_assert(N == 2 || N == 4 || N == 8, "8, 16 or 32 bytes");
    if constexpr (N == 2) {
        const uint2 a = *reinterpret_cast<const uint2 *>(p);
        w[0] = a.x; w[1] = a.y;
    } else {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const uint4 a = reinterpret_cast<const uint4 *>(p)[i];
            w[4 * i] = a.x; w[4 * i + 1] = a.y; w[4 * i + 2] = a.z; w[4 * i + 3] = a.w;
        }
    }
}

template <int D>
__device__ __forceinline__ void load_page(const uint8_t *rec, int lane, RawPage<D> &r) {
    using L = Kv4Page<D>;
    const int n = lane & 15, q = lane >> 4;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        load_words(rec + (16 * s + n) * L::kRow + q * (D / 8), r.k[s]);
        load_words(rec + L::kValues + ((4 * s + q) * 16 + n) * (D / 8), r.v[s]);
    }
    load_words(rec + L::kKeyPairs + lane * (D / 8), r.m);
}

template <int D, bool BF16>
__global__ __launch_bounds__(64 * kWaves) void attn4_kernel(const Attn4Args a) {
    using L = Kv4Page<D>;
    constexpr int NG = L::kGroups, NS = L::kSteps, NT = BF16 ? 1 : 2;
    __shared__ __align__(16) uint32_t pairs[kWaves][2 * D];   // 8 D bytes a page
    __shared__ __align__(16) float o_all[kWaves][kRows][D];
    __shared__ float m_all[kWaves][kRows], l_all[kWaves][kRows];

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int n = lane & 15, quad = lane >> 4;
    const int G = a.heads / a.c.kv_heads;
    int64_t x = blockIdx.x;
    const int split = (int)(x % a.splits);
    x /= a.splits;
    const int kv_head = (int)(x % a.c.kv_heads);
    const Tile t = find_tile(a, x / a.c.kv_heads, G);
    if (t.row0 >= t.rows) return;   // the whole workgroup

    // ---- this lane's row and its query, 8 channels of every 32
    const int64_t row = min(t.row0 + n, t.rows - 1);
    const int64_t token = t.token0 + row / G;
    const int head = kv_head * G + (int)(row % G);
    const int64_t pos = t.pos0 + row / G;
    const int64_t low = a.window > 0 ? pos - a.window + 1 : 0;   // may be negative
    h8 qf[NT][NS];
    float qsum[NG], qs;
    {
        float v[NS][8], top = 0.0f;
#pragma unroll
        for (int j = 0; j < NS; ++j) {
            load8<BF16>(a.q, token * a.q_stride + head * D + 32 * j + 8 * quad, v[j]);
#pragma unroll
            for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[j][e]));
        }
        top = quad_max(top);
        // times 2^k, so that the largest is in [2^9, 2^10)
        const int k = top > 0.0f ? min(10 - __builtin_amdgcn_frexp_expf(top), 126) : 0;
        qs = fmaxf(ldexpf(a.scale_log2, -k), 1.2e-38f);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            float sum = 0.0f;
#pragma unroll
            for (int j = 2 * g; j < 2 * g + 2; ++j) {
                float y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    y[e] = ldexpf(v[j][e], k);
                    sum += y[e];
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float z = y[(e >> 1) + 4 * (e & 1)];
                    const _Float16 hi = (_Float16)z;
                    qf[0][j][e] = hi;
                    if constexpr (NT == 2) qf[NT - 1][j][e] = (_Float16)(z - (float)hi);
                }
            }
            qsum[g] = quad_sum(sum);
        }
    }

    // ---- the pages of this split, every kWaves-th to this wave
    const int64_t i_end = t.pages * (split + 1) / a.splits;
    const int64_t pos_first = t.pos0 + t.row0 / G;
    const int64_t low_last =
        a.window > 0 ? t.pos0 + (min(t.row0 + kRows, t.rows) - 1) / G - a.window + 1 : 0;
    const int32_t *table = a.c.table + t.seq * a.c.max_pages;
    float m = kNoMax, l = 0.0f, omid[NG];
    int E = -14;                 // every step so far is below 2^E
    f4 o[NG][4];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        omid[g] = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[g][i] = f4{0.0f, 0.0f, 0.0f, 0.0f};
    }

    auto page_at = [&](int64_t i) { return i < t.sink_pages ? i : t.first + i - t.sink_pages; };
    for (int64_t i = t.pages * split / a.splits + wave; i < i_end; i += kWaves) {
        const int64_t page = page_at(i), at = table[page], t0 = page * kPage;
        if (at < 0 || at >= a.c.n_pages) continue;   // an absent page
        RawPage<D> r;
        load_page<D>(a.c.cache + (at * a.c.kv_heads + kv_head) * L::kBytes, lane, r);
        // tokens behind the last have pairs of any value
        if (t0 + kPage > t.held) {
            const int left = (int)(t.held - t0);
            if (lane >= 32) {
#pragma unroll
                for (int w = 0; w < D / 32; ++w) {
                    // halfword i of the value pairs: token 4 (i / 8 / NG) + i % 4
                    const int h0 = (lane - 32) * (D / 16) + 2 * w;
                    const int tok = 4 * (h0 / (8 * NG)) + (h0 & 3);
                    if (tok >= left) r.m[w] = 0;
                    else if (tok + 1 >= left) r.m[w] &= 0xffffu;
                }
            }
        }
        // the largest step: lanes 32 on hold four steps, then four middles, and so on
        uint32_t smax = 0;
        if (lane >= 32) {
#pragma unroll
            for (int w = 0; w < D / 32; ++w) {
                const bool steps = D == 64 ? !(lane & 1) : !(w & 2);
                if (steps) smax = max(smax, max(r.m[w] & 0xffffu, r.m[w] >> 16));
            }
        }
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) smax = max(smax, (uint32_t)__shfl_xor((int)smax, d));
        const int E_new = max(E, (int)(smax >> 10) - 14);
        {
            uint32_t *dst = &pairs[wave][lane * (D / 32)];
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
            for (int w = 0; w < D / 32; ++w) dst[w] = r.m[w];
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        }
        // ---- scores of 64 tokens: s[i][e] is token 16 i + 4 quad + e
        float s[4][4], top = -INFINITY;
#pragma unroll
        for (int i4 = 0; i4 < 4; ++i4) {
            const uint32_t *kp = &pairs[wave][(16 * i4 + 4 * quad) * NG];
#pragma unroll
            for (int e = 0; e < 4; ++e) s[i4][e] = 0.0f;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                f4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int j = 2 * g; j < 2 * g + 2; ++j) {
                    h2 c[4];
                    codes8(r.k[i4][j], c);
                    const h8 kf = join(c[0], c[1], c[2], c[3]);
#pragma unroll
                    for (int n2 = 0; n2 < NT; ++n2)
                        acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, qf[n2][j], acc, 0, 0, 0);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const h2 p = as_h2(kp[e * NG + g]);
                    s[i4][e] = fmaf((float)p[0], acc[e], s[i4][e]);
                    s[i4][e] = fmaf((float)p[1], qsum[g], s[i4][e]);
                }
            }
        }
        const bool all_seen = t0 + kPage - 1 <= pos_first && (t0 >= low_last || t0 + kPage <= a.sinks);
        if (!all_seen) {
#pragma unroll
            for (int i4 = 0; i4 < 4; ++i4)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int64_t j = t0 + 16 * i4 + 4 * quad + e;
                    if (j > pos || (j < low && j >= a.sinks)) s[i4][e] = -INFINITY;
                }
        }
#pragma unroll
        for (int i4 = 0; i4 < 4; ++i4)
#pragma unroll
            for (int e = 0; e < 4; ++e) top = fmaxf(top, s[i4][e]);
        const float m_new = fmaxf(m, quad_max(top) * qs);
        if (__any(m_new > m || E_new > E)) {
            const float f = __builtin_amdgcn_exp2f(m - m_new + (float)(E - E_new));
            l *= f;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                omid[g] *= f;
#pragma unroll
                for (int i = 0; i < 4; ++i) o[g][i] *= f;
            }
            m = m_new;
            E = E_new;
        }
        // ---- p * 2^(15 - E), and the second product
        const float ref = m - (float)(15 - E);
#pragma unroll
        for (int i4 = 0; i4 < 4; ++i4)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[i4][e] = __builtin_amdgcn_exp2f(fmaf(s[i4][e], qs, -ref));
                l += s[i4][e];
            }
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                h8 pf[NT];
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const uint32_t *vp =
                        &pairs[wave][D + ((4 * (2 * hf + b) + quad) * NG + g) * 4];
                    const h2 st[2] = {as_h2(vp[0]), as_h2(vp[1])};
                    const h2 md[2] = {as_h2(vp[2]), as_h2(vp[3])};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float p = s[2 * hf + b][e];
                        const float ps = p * (float)st[e >> 1][e & 1];
                        omid[g] = fmaf(p, (float)md[e >> 1][e & 1], omid[g]);
                        const _Float16 hi = (_Float16)ps;
                        pf[0][4 * b + e] = hi;
                        if constexpr (NT == 2)
                            pf[NT - 1][4 * b + e] =
                                (_Float16)fmaf(p, (float)st[e >> 1][e & 1], -(float)hi);
                    }
                }
                h2 c[4][4];   // [two tokens][channel]
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int w = 0; w < 2; ++w) codes8(r.v[2 * hf + b][2 * g + w], c[2 * b + w]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const h8 vf = join(c[0][i], c[1][i], c[2][i], c[3][i]);
#pragma unroll
                    for (int n2 = 0; n2 < NT; ++n2)
                        o[g][i] =
                            __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, pf[n2], o[g][i], 0, 0, 0);
                }
            }
        }
    }

    // ---- join the waves: everything of a row is scaled by 2^-(m + E)
    l = quad_sum(l);
    if (quad == 0) {
        m_all[wave][n] = m + (float)E;
        l_all[wave][n] = l;
    }
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        omid[g] = quad_sum(omid[g]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float4 w;
            w.x = o[g][0][e] + omid[g];
            w.y = o[g][1][e] + omid[g];
            w.z = o[g][2][e] + omid[g];
            w.w = o[g][3][e] + omid[g];
            *reinterpret_cast<float4 *>(&o_all[wave][n][64 * g + 16 * quad + 4 * e]) = w;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kRows * (D / 4); i += 64 * kWaves) {
        const int rr = i / (D / 4), ch = 4 * (i % (D / 4));
        if (t.row0 + rr >= t.rows) continue;
        float top = m_all[0][rr];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) top = fmaxf(top, m_all[w][rr]);
        float sum = 0.0f;
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const float f = __builtin_amdgcn_exp2f(m_all[w][rr] - top);
            const float4 ow = *reinterpret_cast<const float4 *>(&o_all[w][rr][ch]);
            sum = fmaf(f, l_all[w][rr], sum);
            acc.x = fmaf(f, ow.x, acc.x);
            acc.y = fmaf(f, ow.y, acc.y);
            acc.z = fmaf(f, ow.z, acc.z);
            acc.w = fmaf(f, ow.w, acc.w);
        }
        const int64_t rrow = t.row0 + rr;
        const int64_t line = (t.token0 + rrow / G) * a.heads + kv_head * G + rrow % G;
        if (a.splits > 1) {
            const int64_t lines = a.N * a.heads;
            float *part = a.part + ((int64_t)split * lines + line) * (D + 4);
            *reinterpret_cast<float4 *>(part + ch) = acc;
            if (ch == 0) {
                part[D] = top;
                part[D + 1] = sum;
            }
            continue;
        }
        const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
        acc.x *= inv; acc.y *= inv; acc.z *= inv; acc.w *= inv;
        if constexpr (BF16) {
            uint2 w;
            w.x = bf16_bits(acc.x) | bf16_bits(acc.y) << 16;
            w.y = bf16_bits(acc.z) | bf16_bits(acc.w) << 16;
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + line * D + ch) = w;
        } else {
            *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + line * D + ch) = acc;
        }
    }
}

// Joins the splits of a row, in their order: D / 4 lanes to a row.
template <int D, bool BF16>
__global__ __launch_bounds__(256) void attn4_join_kernel(const Attn4Args a) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t line = i / (D / 4), lines = a.N * a.heads;
    const int ch = 4 * (int)(i % (D / 4));
    if (line >= lines || !row_in_call(a.c, line / a.heads)) return;
    const float *part = a.part + line * (D + 4);
    float top = kNoMax;
    for (int s = 0; s < a.splits; ++s) top = fmaxf(top, part[s * lines * (D + 4) + D]);
    float sum = 0.0f;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int s = 0; s < a.splits; ++s) {
        const float *p = part + s * lines * (D + 4);
        const float f = __builtin_amdgcn_exp2f(p[D] - top);
        const float4 ow = *reinterpret_cast<const float4 *>(p + ch);
        sum = fmaf(f, p[D + 1], sum);
        acc.x = fmaf(f, ow.x, acc.x);
        acc.y = fmaf(f, ow.y, acc.y);
        acc.z = fmaf(f, ow.z, acc.z);
        acc.w = fmaf(f, ow.w, acc.w);
    }
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
    acc.x *= inv; acc.y *= inv; acc.z *= inv; acc.w *= inv;
    if constexpr (BF16) {
        uint2 w;
        w.x = bf16_bits(acc.x) | bf16_bits(acc.y) << 16;
        w.y = bf16_bits(acc.z) | bf16_bits(acc.w) << 16;
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + line * D + ch) = w;
    } else {
        *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + line * D + ch) = acc;
    }
}

template <int D, bool BF16>
void launch_d(const Attn4Args &a, hipStream_t st) {
    const int64_t G = a.heads / a.c.kv_heads;
    const int64_t tiles = a.N * G / kRows + a.c.n_seqs;
    hipLaunchKernelGGL((attn4_kernel<D, BF16>),
                       dim3((unsigned)(tiles * a.c.kv_heads * a.splits)), dim3(64 * kWaves), 0, st,
                       a);
    if (a.splits > 1) {
        const int64_t lanes = a.N * a.heads * (D / 4);
        hipLaunchKernelGGL((attn4_join_kernel<D, BF16>), dim3((unsigned)((lanes + 255) / 256)),
                           dim3(256), 0, st, a);
    }
}

}  // namespace

int attn4_splits(int64_t n_seqs, int64_t N, int64_t heads, int64_t kv_heads, int64_t max_kv) {
    // workgroups without a split, and enough splits for four to a compute unit,
    // with at least one page for each wave
    const int64_t tiles = (N * (heads / kv_heads) / kRows + n_seqs) * kv_heads;
    const int64_t pages = (max_kv + kPage - 1) / kPage;
    int64_t s = (4 * 256 + tiles - 1) / tiles;
    if (s > (pages + kWaves - 1) / kWaves) s = (pages + kWaves - 1) / kWaves;
    return s < 1 ? 1 : s > 64 ? 64 : (int)s;
}

hipError_t launch_attn4(const Attn4Args &a, int bf16, int dim, hipStream_t st) {
    if (dim == 64) { if (bf16) launch_d<64, true>(a, st); else launch_d<64, false>(a, st); }
    else if (dim == 128) { if (bf16) launch_d<128, true>(a, st); else launch_d<128, false>(a, st); }
    else { if (bf16) launch_d<256, true>(a, st); else launch_d<256, false>(a, st); }
    return hipGetLastError();
}

}  // namespace bitnet
