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
constexpr int kWanted = 1024;      // workgroups that a launch is split into
constexpr int kMaxSplits = 256;
constexpr float kNoMax = -3.0e38f; // a running maximum before the first visible token

__device__ __forceinline__ h2 as_h2(uint32_t w) { return __builtin_bit_cast(h2, w); }
__device__ __forceinline__ h8 join(h2 a, h2 b, h2 c, h2 d) {
    return h8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// 1024 = 0x6400 twice, in a vector register: with the mask in a scalar one a
// nibble then takes its exponent in a single v_and_or_b32.
__device__ __forceinline__ uint32_t ones_1024() {
    uint32_t w;
    asm("v_mov_b32 %0, 0x64006400" : "=v"(w));
    return w;
}
// Eight nibbles of a word as code - 8, in the order 0 4, 1 5, 2 6, 3 7.  A
// nibble in the low mantissa bits of 1024 makes 1024 + code (or 1024 + 16 code
// one place up); both results are exact.  9 operations for 8 codes.
__device__ __forceinline__ void codes8(uint32_t w, uint32_t one, h2 (&c)[4]) {
    const h2 s = {(_Float16)0.0625f, (_Float16)0.0625f};
    const uint32_t w8 = w >> 8;
    c[0] = as_h2((w & 0x000f000fu) | one) - (_Float16)1032.0f;
    c[1] = as_h2((w & 0x00f000f0u) | one) * s - (_Float16)72.0f;
    c[2] = as_h2((w8 & 0x000f000fu) | one) - (_Float16)1032.0f;
    c[3] = as_h2((w8 & 0x00f000f0u) | one) * s - (_Float16)72.0f;
}
// A zero that the compiler does not know: p * step + zero is then one
// v_fma_mix_f32, which takes the fp16 step without a conversion.
__device__ __forceinline__ float opaque_zero() {
    float z;
    asm("v_mov_b32 %0, 0" : "=v"(z));
    return z;
}

// Over the four lanes that hold a row (l, l ^ 16, l ^ 32, l ^ 48): the swaps
// hand every lane its own and its partner's value.
__device__ __forceinline__ void partners16(float v, float &a, float &b) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false,
                                                    false);
    a = __uint_as_float(r[0]);
    b = __uint_as_float(r[1]);
}
__device__ __forceinline__ void partners32(float v, float &a, float &b) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false,
                                                    false);
    a = __uint_as_float(r[0]);
    b = __uint_as_float(r[1]);
}
__device__ __forceinline__ float quad_max(float v) {
    float a, b;
    partners16(v, a, b);
    partners32(fmaxf(a, b), a, b);
    return fmaxf(a, b);
}
__device__ __forceinline__ float quad_sum(float v) {
    float a, b;
    partners16(v, a, b);
    partners32(a + b, a, b);
    return a + b;
}
// The wave's largest of small non-negative integers, in a scalar register.
__device__ __forceinline__ int wave_max_u16(int v) {
    v = max(v, dpp_i32<kDppXor1>(v));
    v = max(v, dpp_i32<kDppXor2>(v));
    v = max(v, dpp_i32<kDppHalfMirror>(v));
    v = max(v, dpp_i32<kDppMirror>(v));
    v = max(v, dpp_rows_i32<kDppRowBcast15, 0xA>(v));
    v = max(v, dpp_rows_i32<kDppRowBcast31, 0xC>(v));
    return __builtin_amdgcn_readlane(v, 63);
}

// The tile (16 rows of one sequence) that a workgroup works on, and the pages
// its rows see: the first `sink_pages`, then from `first` to the last.
struct Tile {
    int seq, token0, held;      // token0: the sequence's first query token
    uint32_t rows, row0;
    int pos0;                   // position of row 0's token
    int first, sink_pages, pages;
};

__device__ __forceinline__ Tile find_tile(const Attn4Args &a, uint32_t x, uint32_t G) {
    Tile t;
    // the largest b with q_start[b] * G / 16 + b <= x: a sequence has at least
    // as many tiles to itself as its rows need.  64 probes at a time.
    const int lane = threadIdx.x & 63;
    int lo = 0, n = (int)a.c.n_seqs;   // the answer is in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 63) >> 6, b = lo + lane * step;
        const bool ok = lane * step < n && (uint32_t)a.c.q_start[b] * G / kRows + b <= x;
        const int hits = __popcll(__ballot(ok));   // all probes up to the answer's
        const int k = hits > 0 ? hits - 1 : 0;
        lo += k * step;
        n = min(step, n - k * step);
    }
    lo = __builtin_amdgcn_readfirstlane(lo);
    t.seq = lo;
    const int begin = a.c.q_start[lo], end = a.c.q_start[lo + 1];
    t.token0 = begin;
    const bool good = begin >= 0 && end > begin && end <= (int)a.N;
    t.rows = good ? (uint32_t)(end - begin) * G : 0;
    const int tile = (int)(x - ((uint32_t)begin * G / kRows + lo));
    if (tile < 0) t.rows = 0;
    t.row0 = (uint32_t)tile * kRows;
    t.held = (int)held_tokens(a.c, lo);
    t.pos0 = t.held - (end - begin);
    t.pages = t.first = t.sink_pages = 0;
    if (t.row0 >= t.rows) {
        t.rows = 0;
        return t;
    }
    const uint32_t last_row = min(t.row0 + kRows, t.rows) - 1;
    const int pos_a = t.pos0 + (int)(t.row0 / G), pos_b = t.pos0 + (int)(last_row / G);
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

__device__ __forceinline__ void add_part(float4 &acc, float &sum, float f, const float4 &o,
                                         float l) {
    sum = fmaf(f, l, sum);
    acc.x = fmaf(f, o.x, acc.x);
    acc.y = fmaf(f, o.y, acc.y);
    acc.z = fmaf(f, o.z, acc.z);
    acc.w = fmaf(f, o.w, acc.w);
}
// Four channels of a finished row; a row that saw nothing has no sum.
template <bool BF16>
__device__ __forceinline__ void store_out(void *out, int64_t at, float4 acc, float sum) {
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
    acc.x *= inv; acc.y *= inv; acc.z *= inv; acc.w *= inv;
    if constexpr (BF16) {
        uint2 w;
        w.x = bf16_bits(acc.x) | bf16_bits(acc.y) << 16;
        w.y = bf16_bits(acc.z) | bf16_bits(acc.w) << 16;
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(out) + at) = w;
    } else {
        *reinterpret_cast<float4 *>(static_cast<float *>(out) + at) = acc;
    }
}

// What a wave carries along its pages.
template <int D, int NT>
struct Running {
    float m, l, omid[D / 64];   // maximum, sum of p and of p * middle, of this lane's tokens
    int E;                      // every step so far is below 2^E
    f4 o[D / 64][4];            // channel 64 g + 16 quad + 4 e + i of o[g][i][e]
};

template <int D, bool BF16>
__global__ __launch_bounds__(64 * kWaves, D == 256 ? 1 : 2) void attn4_kernel(const Attn4Args a) {
    using L = Kv4Page<D>;
    constexpr int NG = L::kGroups, NS = L::kSteps, NT = BF16 ? 1 : 2;
    __shared__ __align__(16) uint32_t pairs[kWaves][2 * D];   // 8 D bytes a page
    __shared__ __align__(16) float o_all[kWaves][kRows][D];
    __shared__ float m_all[kWaves][kRows], l_all[kWaves][kRows];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, quad = lane >> 4;
    const uint32_t G = (uint32_t)a.heads / (uint32_t)a.c.kv_heads;
    const int kv_head = blockIdx.y, split = blockIdx.z;
    const Tile t = find_tile(a, blockIdx.x, G);
    if (t.rows == 0) return;   // the whole workgroup
    const uint32_t one = ones_1024();
    const float zero = opaque_zero();

    // ---- this lane's row and its query, 8 channels of every 32
    const uint32_t row = min(t.row0 + n, t.rows - 1), row_tok = row / G;
    const int head = kv_head * (int)G + (int)(row - row_tok * G);
    const int pos = t.pos0 + (int)row_tok;
    const int low = a.window > 0 ? pos - a.window + 1 : 0;   // may be negative
    h8 qf[NT][NS];
    float qsum[NG], qs;
    {
        float v[NS][8], top = 0.0f;
        const int64_t at = (int64_t)(t.token0 + (int)row_tok) * a.q_stride + head * D + 8 * quad;
#pragma unroll
        for (int j = 0; j < NS; ++j) load8<BF16>(a.q, at + 32 * j, v[j]);
#pragma unroll
        for (int j = 0; j < NS; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[j][e]));
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
    const int i0 = (int)((uint32_t)t.pages * split / a.splits) + wave;
    const int i_end = (int)((uint32_t)t.pages * (split + 1) / a.splits);
    const int pos_first = t.pos0 + (int)(t.row0 / G);
    const int low_last = a.window > 0
                             ? t.pos0 + (int)((min(t.row0 + kRows, t.rows) - 1) / G) - a.window + 1
                             : 0;
    const int32_t *table = a.c.table + (int64_t)t.seq * a.c.max_pages;
    auto page_at = [&](int i) { return i < t.sink_pages ? i : t.first + i - t.sink_pages; };
    const uint8_t *cache = a.c.cache + (int64_t)kv_head * L::kBytes;
    const int64_t page_bytes = (int64_t)a.c.kv_heads * L::kBytes;

    Running<D, NT> R;
    R.m = kNoMax;
    R.l = 0.0f;
    R.E = -14;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        R.omid[g] = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) R.o[g][i] = f4{0.0f, 0.0f, 0.0f, 0.0f};
    }

    auto process = [&](int i, RawPage<D> &r) {
        const int t0 = page_at(i) * kPage;
        // tokens behind the last have pairs of any value
        if (t0 + kPage > t.held) {
            const int left = t.held - t0;
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
#pragma unroll
        for (int w = 0; w < D / 32; ++w)
            if (D == 64 || !(w & 2)) smax = max(smax, max(r.m[w] & 0xffffu, r.m[w] >> 16));
        if (lane < 32 || (D == 64 && (lane & 1))) smax = 0;
        const int E_new = max(R.E, (wave_max_u16((int)smax) >> 10) - 14);
        {
            uint32_t *dst = &pairs[wave][lane * (D / 32)];
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
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
            for (int g = 0; g < NG; ++g) {
                f4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int j = 2 * g; j < 2 * g + 2; ++j) {
                    h2 c[4];
                    codes8(r.k[i4][j], one, c);
                    const h8 kf = join(c[0], c[1], c[2], c[3]);
#pragma unroll
                    for (int n2 = 0; n2 < NT; ++n2)
                        acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, qf[n2][j], acc, 0, 0, 0);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const h2 p = as_h2(kp[e * NG + g]);
                    const float b = g == 0 ? (float)p[1] * qsum[0]
                                           : fmaf((float)p[1], qsum[g], s[i4][e]);
                    s[i4][e] = fmaf((float)p[0], acc[e], b);
                }
            }
        }
        const bool all_seen =
            t0 + kPage - 1 <= pos_first && (t0 >= low_last || t0 + kPage <= a.sinks);
        if (!all_seen) {
#pragma unroll
            for (int i4 = 0; i4 < 4; ++i4)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = t0 + 16 * i4 + 4 * quad + e;
                    const bool hidden = (j > pos) | ((j < low) & (j >= a.sinks));
                    s[i4][e] = hidden ? -INFINITY : s[i4][e];
                }
        }
#pragma unroll
        for (int i4 = 0; i4 < 4; ++i4)
#pragma unroll
            for (int e = 0; e < 4; ++e) top = fmaxf(top, s[i4][e]);
        const float m_new = fmaxf(R.m, quad_max(top) * qs);
        if (E_new > R.E || __any(m_new > R.m)) {
            const float f = __builtin_amdgcn_exp2f(R.m - m_new + (float)(R.E - E_new));
            R.l *= f;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                R.omid[g] *= f;
#pragma unroll
                for (int i = 0; i < 4; ++i) R.o[g][i] *= f;
            }
            R.m = m_new;
            R.E = E_new;
        }
        // ---- p * 2^(15 - E), and the second product
        const float ref = R.m - (float)(15 - R.E);
#pragma unroll
        for (int i4 = 0; i4 < 4; ++i4)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[i4][e] = __builtin_amdgcn_exp2f(fmaf(s[i4][e], qs, -ref));
                R.l += s[i4][e];
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
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        const float p0 = s[2 * hf + b][2 * w], p1 = s[2 * hf + b][2 * w + 1];
                        const h2 md = as_h2(vp[2 + w]);
                        R.omid[g] = fmaf(p0, (float)md[0], R.omid[g]);
                        R.omid[g] = fmaf(p1, (float)md[1], R.omid[g]);
                        const h2 st = as_h2(vp[w]);
                        const h2 hi = {(_Float16)fmaf(p0, (float)st[0], zero),
                                       (_Float16)fmaf(p1, (float)st[1], zero)};
                        pf[0][4 * b + 2 * w] = hi[0];
                        pf[0][4 * b + 2 * w + 1] = hi[1];
                        if constexpr (NT == 2) {
                            pf[NT - 1][4 * b + 2 * w] =
                                (_Float16)fmaf(p0, (float)st[0], -(float)hi[0]);
                            pf[NT - 1][4 * b + 2 * w + 1] =
                                (_Float16)fmaf(p1, (float)st[1], -(float)hi[1]);
                        }
                    }
                }
                h2 c[4][4];   // [two tokens][channel]
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int w = 0; w < 2; ++w)
                        codes8(r.v[2 * hf + b][2 * g + w], one, c[2 * b + w]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const h8 vf = join(c[0][i], c[1][i], c[2][i], c[3][i]);
#pragma unroll
                    for (int n2 = 0; n2 < NT; ++n2)
                        R.o[g][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, pf[n2], R.o[g][i],
                                                                           0, 0, 0);
                }
            }
        }
    };

    // 64 table entries at a time, one a lane, with a bit for each page that is
    // there; they are waited for before the pages, so that no wait of the inner
    // loop takes in the page that is on its way while another is worked on.  For
    // the same reason a page is always loaded, at the end the last one again
    // (from the L2): the count of loads in flight is then the same on every path.
    // At 256 channels two pages and the accumulators are more than a wave's
    // registers.
    for (int from = i0; from < i_end; from += 64 * kWaves) {
        const int mine = from + kWaves * lane;
        const int ids = mine < i_end ? table[page_at(mine)] : -1;
        uint64_t there = __ballot(ids >= 0 && ids < a.c.n_pages);
        int j = 0;
        bool more = there != 0;
        if (!more) continue;
        auto fetch = [&](RawPage<D> &r) {   // the next page; its index
            more = there != 0;
            if (more) j = __builtin_ctzll(there);
            there &= there - 1;
            load_page<D>(cache + __builtin_amdgcn_readlane(ids, j) * page_bytes, lane, r);
            return from + kWaves * j;
        };
        RawPage<D> ra;
        int i = fetch(ra);
        if constexpr (D < 256) {
            RawPage<D> rb;
            while (true) {
                const int i2 = fetch(rb);
                process(i, ra);
                if (!more) break;
                i = fetch(ra);
                process(i2, rb);
                if (!more) break;
            }
        } else {
            while (true) {
                process(i, ra);
                if (there == 0) break;
                i = fetch(ra);
            }
        }
    }

    // ---- join the waves: everything of a row is scaled by 2^-(m + E)
    R.l = quad_sum(R.l);
    if (quad == 0) {
        m_all[wave][n] = R.m + (float)R.E;
        l_all[wave][n] = R.l;
    }
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        const float omid = quad_sum(R.omid[g]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float4 w;
            w.x = R.o[g][0][e] + omid;
            w.y = R.o[g][1][e] + omid;
            w.z = R.o[g][2][e] + omid;
            w.w = R.o[g][3][e] + omid;
            *reinterpret_cast<float4 *>(&o_all[wave][n][64 * g + 16 * quad + 4 * e]) = w;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kRows * (D / 4); i += 64 * kWaves) {
        const int rr = i / (D / 4), ch = 4 * (i % (D / 4));
        const uint32_t rrow = t.row0 + rr, tok = rrow / G;
        if (rrow >= t.rows) continue;
        float top = m_all[0][rr];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) top = fmaxf(top, m_all[w][rr]);
        float sum = 0.0f;
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
            add_part(acc, sum, __builtin_amdgcn_exp2f(m_all[w][rr] - top),
                     *reinterpret_cast<const float4 *>(&o_all[w][rr][ch]), l_all[w][rr]);
        const int64_t line =
            (int64_t)(t.token0 + (int)tok) * a.heads + kv_head * G + (rrow - tok * G);
        if (a.splits > 1) {
            float *part = a.part + ((int64_t)split * a.N * a.heads + line) * (D + 4);
            *reinterpret_cast<float4 *>(part + ch) = acc;
            if (ch == 0) {
                part[D] = top;
                part[D + 1] = sum;
            }
        } else {
            store_out<BF16>(a.out, line * D + ch, acc, sum);
        }
    }
}

// Joins the splits of a row: D / 4 lanes to its channels, `par` (a power of
// two) groups of them to its splits, always added in the same order.
template <int D, bool BF16>
__global__ __launch_bounds__(256) void attn4_join_kernel(const Attn4Args a, int par) {
    constexpr int kLanes = D / 4, kSlots = 256 / kLanes;
    __shared__ float4 o_all[256];
    __shared__ float m_all[kSlots], l_all[kSlots];
    const int slot = threadIdx.x / kLanes, ch = 4 * (threadIdx.x % kLanes);
    const int g = slot & (par - 1);
    const int64_t line = (int64_t)blockIdx.x * (kSlots / par) + slot / par, lines = a.N * a.heads;
    const bool mine = line < lines && row_in_call(a.c, line / a.heads);
    const float *part = a.part + line * (D + 4);
    const int64_t stride = lines * (D + 4);
    float top = kNoMax, sum = 0.0f;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (mine) {
        for (int s = g; s < a.splits; s += par) top = fmaxf(top, part[s * stride + D]);
#pragma unroll 4
        for (int s = g; s < a.splits; s += par) {
            const float *p = part + s * stride;
            add_part(acc, sum, __builtin_amdgcn_exp2f(p[D] - top),
                     *reinterpret_cast<const float4 *>(p + ch), p[D + 1]);
        }
    }
    if (par > 1) {
        o_all[threadIdx.x] = acc;
        if (ch == 0) {
            m_all[slot] = top;
            l_all[slot] = sum;
        }
        __syncthreads();
        if (g != 0 || !mine) return;
        for (int i = 1; i < par; ++i) top = fmaxf(top, m_all[slot + i]);
        sum = 0.0f;
        acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int i = 0; i < par; ++i)
            add_part(acc, sum, __builtin_amdgcn_exp2f(m_all[slot + i] - top),
                     o_all[threadIdx.x + i * kLanes], l_all[slot + i]);
    }
    if (mine) store_out<BF16>(a.out, line * D + ch, acc, sum);
}

template <int D, bool BF16>
void launch_d(const Attn4Args &a, hipStream_t st) {
    const int64_t G = a.heads / a.c.kv_heads;
    const int64_t tiles = a.N * G / kRows + a.c.n_seqs;
    hipLaunchKernelGGL((attn4_kernel<D, BF16>),
                       dim3((unsigned)tiles, (unsigned)a.c.kv_heads, (unsigned)a.splits),
                       dim3(64 * kWaves), 0, st, a);
    if (a.splits > 1) {
        constexpr int kSlots = 256 / (D / 4);
        int par = 1;
        while (par < kSlots && 2 * par < a.splits) par *= 2;
        const int64_t lines = a.N * a.heads, per = kSlots / par;
        hipLaunchKernelGGL((attn4_join_kernel<D, BF16>),
                           dim3((unsigned)((lines + per - 1) / per)), dim3(256), 0, st, a, par);
    }
}

}  // namespace

int attn4_splits(int64_t n_seqs, int64_t N, int64_t heads, int64_t kv_heads, int64_t max_kv) {
    // workgroups without a split, and enough splits for four to a compute unit,
    // with at least one page for each wave
    const int64_t tiles = (N * (heads / kv_heads) / kRows + n_seqs) * kv_heads;
    const int64_t pages = (max_kv + kPage - 1) / kPage;
    int64_t s = (kWanted + tiles - 1) / tiles;
    if (s > (pages + kWaves - 1) / kWaves) s = (pages + kWaves - 1) / kWaves;
    return s < 1 ? 1 : s > kMaxSplits ? kMaxSplits : (int)s;
}

hipError_t launch_attn4(const Attn4Args &a, int bf16, int dim, hipStream_t st) {
    if (dim == 64) { if (bf16) launch_d<64, true>(a, st); else launch_d<64, false>(a, st); }
    else if (dim == 128) { if (bf16) launch_d<128, true>(a, st); else launch_d<128, false>(a, st); }
    else { if (bf16) launch_d<256, true>(a, st); else launch_d<256, false>(a, st); }
    return hipGetLastError();
}

}  // namespace bitnet
