// attn_kv4.hip -- causal attention over the 4-bit cache (kv4.h: its layout),
// with an optional sliding window and a few first tokens that stay visible.
//
//   out[row] = sum_t p_t v_t / sum_t p_t,   p_t = 2^(x_t - max x),
//   x_t = log2(e) * scale * q . k_t
// in one pass over the pages with a running maximum.  The queries of all heads
// that share a kv head are rows of one problem: row r of a sequence is token
// r / G, head r % G of the group.
//
// Both products run on the fp16 16x16x32 matrix instruction with the codes in
// place of the values.  For a group of 64 channels, value = mid + step * (code - 8):
//   q . k_t       = sum_g step_tg (q_g . (code_tg - 8)) + mid_tg sum(q_g)
//   sum_t p_t v_t = sum_t (p_t step_tg) (code_tg - 8)   + sum_t p_t mid_tg
// The second terms are matrix products too, of the pairs as they are stored with
// the sums of q and with p; a row of ones among them gives sum p.
//   bf16 calls take the nibbles as they are: in the low bits of an fp16 a nibble is
// the subnormal number code * 2^-24 (or 16 times that, one nibble up), which the
// instruction takes, at five operations for eight codes; the 8 moves into the
// second terms.  Its sums are then good to about 2^-17 (it aligns a subnormal's
// product by the smallest normal exponent), far below what a bf16 result holds.
//   fp32 calls make code - 8 a normal number, exactly, at nine operations.
// q is scaled by a power of two per row, p * step by one per page (from the
// largest step met so far, tracked like the maximum), so neither leaves fp16's
// normal range; bf16 calls round q (8 bits), p and p * step once to fp16's 11 bits,
// finer than the output, fp32 calls carry them as two fp16 terms (22 bits).  Sums,
// maxima and accumulators are fp32.
//
// The first product is taken transposed (tokens x rows), which leaves a lane
// with 16 tokens of one row: that is exactly the fragment that the second
// product (channels x rows) takes, so p never crosses lanes, and the running
// maximum and the accumulators of a row all live in the same lanes.
#include <algorithm>

#include "kv4.h"

namespace bitnet {

namespace {

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));

constexpr int kRows = 16;          // rows of a tile
constexpr int kWaves = 4;          // waves of a workgroup; each takes every fourth page
constexpr int kWanted = 512;      // workgroups that a launch is split into
constexpr int kMaxSplits = 256;
constexpr int kPromptFrom = 64;   // rows of a sequence, on average
constexpr int kPromptChunk = 16;
constexpr int kJoinThreads = 1024;
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
// The eight codes of a word in the order 0 4, 1 5, 2 6, 3 7.  RAW: as fp16
// subnormals code * 2^-24, the second and fourth pair 16 times as large.  Else
// code - 8: a nibble in the low mantissa bits of 1024 makes 1024 + code (or 1024
// + 16 code one place up), and one packed operation the rest, exactly.
template <bool RAW>
__device__ __forceinline__ void codes8(uint32_t w, uint32_t one, h2 (&c)[4]) {
    const uint32_t w8 = w >> 8;
    if constexpr (RAW) {
        c[0] = as_h2(w & 0x000f000fu);
        c[1] = as_h2(w & 0x00f000f0u);
        c[2] = as_h2(w8 & 0x000f000fu);
        c[3] = as_h2(w8 & 0x00f000f0u);
    } else {
        const h2 s = {(_Float16)0.0625f, (_Float16)0.0625f};
        c[0] = as_h2((w & 0x000f000fu) | one) - (_Float16)1032.0f;
        c[1] = as_h2((w & 0x00f000f0u) | one) * s - (_Float16)72.0f;
        c[2] = as_h2((w8 & 0x000f000fu) | one) - (_Float16)1032.0f;
        c[3] = as_h2((w8 & 0x00f000f0u) | one) * s - (_Float16)72.0f;
    }
}
__device__ __forceinline__ f4 mfma(h8 a, h8 b, f4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
// 2^e as fp16, -24 <= e <= 15.
__device__ __forceinline__ _Float16 pow2_f16(int e) {
    return __builtin_bit_cast(_Float16, (uint16_t)(e >= -14 ? (e + 15) << 10 : 1 << (e + 24)));
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

// The tile (ROWS rows of one sequence) that a workgroup works on, and the pages
// its rows see: the first `sink_pages`, then from `first` to the last.
struct Tile {
    int seq, token0, held;      // token0: the sequence's first query token
    uint32_t rows, row0;
    int pos0;                   // position of row 0's token
    int first, sink_pages, pages;
};

template <int ROWS>
__device__ __forceinline__ Tile find_tile(const Attn4Args &a, uint32_t x, uint32_t G) {
    Tile t;
    // the largest b with q_start[b] * G / ROWS + b <= x: a sequence has at least
    // as many tiles to itself as its rows need.  64 probes at a time.
    const int lane = threadIdx.x & 63;
    int lo = 0, n = (int)a.c.n_seqs;   // the answer is in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 63) >> 6, b = lo + lane * step;
        const bool ok = lane * step < n && (uint32_t)a.c.q_start[b] * G / ROWS + b <= x;
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
    const int tile = (int)(x - ((uint32_t)begin * G / ROWS + lo));
    if (tile < 0) t.rows = 0;
    t.row0 = (uint32_t)tile * ROWS;
    t.held = (int)held_tokens(a.c, lo);
    t.pos0 = t.held - (end - begin);
    t.pages = t.first = t.sink_pages = 0;
    if (t.row0 >= t.rows) {
        t.rows = 0;
        return t;
    }
    const uint32_t last_row = min(t.row0 + ROWS, t.rows) - 1;
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

// A row's query as the first product takes it, 8 channels of every 32 in this
// lane, times 2^k; what its result is multiplied by to give a power of two's
// exponent; and the sums of q that stand against a token's (step, middle).  RAW:
// the product's codes are subnormal.
template <int D, bool BF16, bool RAW>
__device__ __forceinline__ void load_query(const Attn4Args &a, int token, int head, int quad,
                                           h8 (&qf)[BF16 ? 1 : 2][D / 32], h8 &cf, float &qs) {
    float v[D / 32][8], top = 0.0f;
    const int64_t at = token * a.q_stride + head * D + 8 * quad;
#pragma unroll
    for (int j = 0; j < D / 32; ++j) load8<BF16>(a.q, at + 32 * j, v[j]);
#pragma unroll
    for (int j = 0; j < D / 32; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[j][e]));
    top = quad_max(top);
    // q times 2^k: the largest is in [2^14, 2^15); the sums of q times 2^(k - 11):
    // the largest they can be is 2^10
    const int k = top > 0.0f ? min(15 - __builtin_amdgcn_frexp_expf(top), 140) : 0;
    qs = fmaxf(ldexpf(a.scale_log2, (RAW ? 24 : 0) - k), 1.2e-38f);
    cf = h8{0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int g = 0; g < D / 64; ++g) {
        float sum = 0.0f;
#pragma unroll
        for (int j = 2 * g; j < 2 * g + 2; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int ch = (e >> 1) + 4 * (e & 1);
                sum += ldexpf(v[j][ch], k - 11);
                const float z = ldexpf(v[j][ch], k - (RAW && (e & 2) ? 4 : 0));
                const _Float16 hi = (_Float16)z;
                qf[0][j][e] = hi;
                if constexpr (!BF16) qf[1][j][e] = (_Float16)(z - (float)hi);
            }
        sum = quad_sum(sum);
        // -8 (raw codes) and 1 times the sum, its upper term in the first 8 of 32
        // places and its lower in the next
        const _Float16 hi = (_Float16)sum;
        const _Float16 part = quad == 0   ? hi
                              : quad == 1 ? (_Float16)(sum - (float)hi)
                                          : (_Float16)0.0f;
        cf[2 * g] = RAW ? (_Float16)-8.0f * part : (_Float16)0.0f;
        cf[2 * g + 1] = part;
    }
}

template <int D, bool BF16>
__global__ __launch_bounds__(64 * kWaves, D == 256 ? 1 : 2) void attn4_kernel(const Attn4Args a) {
    using L = Kv4Page<D>;
    constexpr int NG = L::kGroups, NS = L::kSteps, NT = BF16 ? 1 : 2;
    constexpr int kCodeExp = BF16 ? 24 : 0;   // raw codes carry 2^-24, and every second pair 16
    __shared__ __align__(16) uint32_t pairs[kWaves][2 * D];   // 8 D bytes a page
    __shared__ __align__(16) uint32_t ones[2];                // four fp16 ones
    __shared__ __align__(16) float o_all[kWaves][kRows][D];
    __shared__ float m_all[kWaves][kRows], l_all[kWaves][kRows];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, quad = lane >> 4;
    const uint32_t G = (uint32_t)a.heads / (uint32_t)a.c.kv_heads;
    // heads first: with eight of them a head's tiles share an XCD and its L2
    const uint32_t x = blockIdx.x / (uint32_t)a.c.kv_heads;
    const int kv_head = (int)(blockIdx.x - x * a.c.kv_heads);
    const uint32_t tile = x / (uint32_t)a.splits;
    const int split = (int)(x - tile * a.splits);
    const Tile t = find_tile<kRows>(a, tile, G);
    if (t.rows == 0) return;   // the whole workgroup
    const int i_begin = min(split * a.chunk, t.pages);
    const int i_end = split == a.splits - 1 ? t.pages : min(i_begin + a.chunk, t.pages);
    if (a.splits > 1 && i_begin == i_end) {   // nothing here: parts without a sum
        if (threadIdx.x < kRows && t.row0 + threadIdx.x < t.rows) {
            const uint32_t r = t.row0 + threadIdx.x, tok = r / G;
            const int64_t line = (int64_t)(t.token0 + (int)tok) * a.heads + kv_head * G + (r - tok * G);
            float *part = a.part + ((int64_t)split * a.N * a.heads + line) * (D + 4);
            part[D + 1] = 0.0f;
        }
        return;
    }

    // ---- the pages of this split, every kWaves-th to this wave.  64 table entries
    // at a time, one a lane, with a bit for each page that is there; they are
    // waited for before the pages, so that no wait of the inner loop takes in the
    // page that is on its way while another is worked on.  For the same reason a
    // page is always loaded, at the end the last one again (from the L2): the
    // count of loads in flight is then the same on every path.
    const int32_t *table = a.c.table + (int64_t)t.seq * a.c.max_pages;
    auto page_at = [&](int i) { return i < t.sink_pages ? i : t.first + i - t.sink_pages; };
    const uint8_t *cache = a.c.cache + (int64_t)kv_head * L::kBytes;
    const int64_t page_bytes = (int64_t)a.c.kv_heads * L::kBytes;
    int from = i_begin + wave, ids = -1, id = 0, at_bit = 0;
    uint64_t there = 0;
    bool more = false;   // whether the page fetched last is one to work on
    auto load_ids = [&]() {
        const int mine = from + kWaves * lane;
        ids = mine < i_end ? table[page_at(mine)] : -1;
        there = __ballot(ids >= 0 && ids < a.c.n_pages);
    };
    auto fetch = [&](RawPage<D> &r) {
        more = there != 0;
        if (more) {
            at_bit = __builtin_ctzll(there);
            there &= there - 1;
            id = __builtin_amdgcn_readlane(ids, at_bit);
        }
        load_page<D>(cache + id * page_bytes, lane, r);
        return from + kWaves * at_bit;
    };
    RawPage<D> ra;
    load_ids();
    int i = fetch(ra);

    const uint32_t one = BF16 ? 0 : ones_1024();
    // ---- this lane's row and its query, 8 channels of every 32
    const uint32_t row = min(t.row0 + n, t.rows - 1), row_tok = row / G;
    const int head = kv_head * (int)G + (int)(row - row_tok * G);
    const int pos = t.pos0 + (int)row_tok;
    const int low = a.window > 0 ? pos - a.window + 1 : 0;   // may be negative
    h8 qf[NT][NS], cf;
    float qs;
    load_query<D, BF16, BF16>(a, t.token0 + (int)row_tok, head, quad, qf, cf, qs);

    const int pos_first = t.pos0 + (int)(t.row0 / G);
    const int low_last = a.window > 0
                             ? t.pos0 + (int)((min(t.row0 + kRows, t.rows) - 1) / G) - a.window + 1
                             : 0;

    // What is carried along the pages.  The weights p are 2^(x - m + 15), the
    // steps in front of the second product are divided by 2^E.  `sums` is the product of p with what row n of 16 stands for:
    // row 2 g the steps of group g, 2 g + 1 its middles, 2 NG + 1 ones.
    float m = kNoMax;
    int E = -14;                 // every step so far is below 2^E
    f4 o[NG][4], sums = {0.0f, 0.0f, 0.0f, 0.0f};   // o[g][i][e]: channel 64 g + 16 quad + 4 e + i
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[g][i] = f4{0.0f, 0.0f, 0.0f, 0.0f};
    if (threadIdx.x < 2) ones[threadIdx.x] = 0x3c003c00u;
    __syncthreads();
    const uint32_t *sums_from[4];   // this lane's row of `sums`, for tokens 16 i + 4 quad ..
#pragma unroll
    for (int i = 0; i < 4; ++i)
        sums_from[i] = n == 2 * NG + 1
                           ? ones
                           : &pairs[wave][D + (4 * i + quad) * NG * 4 + 2 * (n & (2 * NG - 1))];

    auto process = [&](int at, RawPage<D> &r) {
        const int t0 = page_at(at) * kPage;
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
        const bool steps_here = lane >= 32 && (D > 64 || !(lane & 1));
        uint32_t smax = 0;
#pragma unroll
        for (int w = 0; w < D / 32; ++w)
            if (D == 64 || !(w & 2)) smax = max(smax, max(r.m[w] & 0xffffu, r.m[w] >> 16));
        const int E_new = max(E, (wave_max_u16(steps_here ? (int)smax : 0) >> 10) - 14);
        {
            const _Float16 f = steps_here ? pow2_f16(-E_new) : (_Float16)1.0f;
            uint32_t *dst = &pairs[wave][lane * (D / 32)];
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int w = 0; w < D / 32; ++w)
                dst[w] = D == 64 || !(w & 2) ? __builtin_bit_cast(uint32_t, as_h2(r.m[w]) * f)
                                             : r.m[w];
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        }
        // ---- scores of 64 tokens: s[i][e] is token 16 i + 4 quad + e
        float s[4][4], top = -INFINITY;
#pragma unroll
        for (int i4 = 0; i4 < 4; ++i4) {
            h8 pf = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const h2 p = as_h2(pairs[wave][(16 * i4 + n) * NG + g]);
                pf[2 * g] = p[0];
                pf[2 * g + 1] = p[1];
            }
            const f4 rest = mfma(pf, cf, f4{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
            for (int e = 0; e < 4; ++e) s[i4][e] = rest[e] * (BF16 ? 0x1p-13f : 0x1p11f);
            const uint32_t *kp = &pairs[wave][(16 * i4 + 4 * quad) * NG];
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                f4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int j = 2 * g; j < 2 * g + 2; ++j) {
                    h2 c[4];
                    codes8<BF16>(r.k[i4][j], one, c);
#pragma unroll
                    for (int n2 = 0; n2 < NT; ++n2)
                        acc = mfma(join(c[0], c[1], c[2], c[3]), qf[n2][j], acc);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    s[i4][e] = fmaf((float)as_h2(kp[e * NG + g])[0], acc[e], s[i4][e]);
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
        const float m_new = fmaxf(m, quad_max(top) * qs);
        if (E_new > E || __any(m_new > m)) {
            const float f = __builtin_amdgcn_exp2f(m - m_new), fs = ldexpf(f, E - E_new);
            sums[0] *= fs;
            sums[1] *= f;
            sums[2] *= fs;
            sums[3] *= f;
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[g][i] *= fs;
            m = m_new;
            E = E_new;
        }
        // ---- p, and the second product
        const float ref = m - 15.0f;
#pragma unroll
        for (int i4 = 0; i4 < 4; ++i4)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                s[i4][e] = __builtin_amdgcn_exp2f(fmaf(s[i4][e], qs, -ref));
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            h2 p[NT][4];   // pairs of tokens: two of subtile 2 hf, two of 2 hf + 1
            h2 from[4];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const float p0 = s[2 * hf + (w >> 1)][2 * (w & 1)];
                const float p1 = s[2 * hf + (w >> 1)][2 * (w & 1) + 1];
                p[0][w] = h2{(_Float16)p0, (_Float16)p1};
                if constexpr (NT == 2)
                    p[NT - 1][w] = h2{(_Float16)(p0 - (float)p[0][w][0]),
                                      (_Float16)(p1 - (float)p[0][w][1])};
                from[w] = as_h2(sums_from[2 * hf + (w >> 1)][w & 1]);
            }
#pragma unroll
            for (int n2 = 0; n2 < NT; ++n2)
                sums = mfma(join(from[0], from[1], from[2], from[3]),
                            join(p[n2][0], p[n2][1], p[n2][2], p[n2][3]), sums);
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                h2 ps[NT][4], c[4][4];   // p * step, and the codes [two tokens][channel]
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const h2 st = as_h2(
                        pairs[wave][D + ((4 * (2 * hf + (w >> 1)) + quad) * NG + g) * 4 + (w & 1)]);
                    ps[0][w] = p[0][w] * st;
                    if constexpr (NT == 2)
                        ps[NT - 1][w] = __builtin_elementwise_fma(
                            p[NT - 1][w], st, __builtin_elementwise_fma(p[0][w], st, -ps[0][w]));
                    codes8<BF16>(r.v[2 * hf + (w >> 1)][2 * g + (w & 1)], one, c[w]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int n2 = 0; n2 < NT; ++n2)
                        o[g][i] = mfma(join(c[0][i], c[1][i], c[2][i], c[3][i]),
                                       join(ps[n2][0], ps[n2][1], ps[n2][2], ps[n2][3]), o[g][i]);
            }
        }
    };

    while (true) {
        if constexpr (D * NT < 256) {
            RawPage<D> rb;
            while (more) {
                const int i2 = fetch(rb);
                process(i, ra);
                if (!more) break;
                i = fetch(ra);
                process(i2, rb);
            }
        } else {   // two pages and the rest are more than a wave's registers
            while (more) {
                process(i, ra);
                i = fetch(ra);
            }
        }
        from += 64 * kWaves;
        if (from >= i_end) break;
        load_ids();
        i = fetch(ra);
    }

    // ---- join the waves: everything of a row is scaled by 2^(15 - m)
    auto sum_row = [&](int r) { return __shfl(sums[r & 3], n + 16 * (r >> 2)); };
    const float l = sum_row(2 * NG + 1), up = ldexpf(1.0f, kCodeExp + E);
    const float up1 = BF16 ? up * 0.0625f : up;
    if (quad == 0) {
        m_all[wave][n] = m;
        l_all[wave][n] = l;
    }
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        float rest = sum_row(2 * g + 1);
        if (BF16) rest -= sum_row(2 * g) * ldexpf(8.0f, E);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float4 w;
            w.x = fmaf(o[g][0][e], up, rest);
            w.y = fmaf(o[g][1][e], up1, rest);
            w.z = fmaf(o[g][2][e], up, rest);
            w.w = fmaf(o[g][3][e], up1, rest);
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

// Prompts: a workgroup takes kPromptRows rows, and its waves share each page
// through LDS.  A page's codes become matrix fragments once, a quarter by each
// wave, while the page before it is worked on: bf16 calls make them the values
// themselves (one fp16 rounding, 11 bits), so a score needs nothing but the mask
// and the exponential after its product; fp32 calls make them code - 8 and apply
// the pairs as attn4_kernel does.
template <int D, bool BF16>
struct Prompt {
    static constexpr int kRt = D == 64 ? (BF16 ? 4 : 2) : D == 128 && BF16 ? 2 : 1;
    static constexpr int kRows = 64 * kRt;   // 16 * kRt rows to each of four waves
};

// One page's codes and pairs as a wave loads its quarter: 16 tokens of the keys,
// and for the values the units (32 tokens, group) u = wave, wave + 4, ..
template <int D>
struct RawQuarter {
    static constexpr int kUnits = D == 64 ? 1 : D / 128;
    uint32_t k[D / 32], kp[D / 64];
    uint32_t v[kUnits][2][2], vp[kUnits][2][4];
};
template <int D>
__device__ __forceinline__ void load_quarter(const uint8_t *rec, int lane, int wave,
                                             RawQuarter<D> &r) {
    using L = Kv4Page<D>;
    const int n = lane & 15, q = lane >> 4;
    load_words(rec + (16 * wave + n) * L::kRow + q * (D / 8), r.k);
    const uint32_t *kp =
        reinterpret_cast<const uint32_t *>(rec + L::kKeyPairs) + (16 * wave + n) * L::kGroups;
#pragma unroll
    for (int g = 0; g < L::kGroups; ++g) r.kp[g] = kp[g];
#pragma unroll
    for (int i = 0; i < RawQuarter<D>::kUnits; ++i) {
        const int u = (wave + 4 * i) % (2 * L::kGroups), hf = u / L::kGroups, g = u % L::kGroups;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int blk = 4 * (2 * hf + b) + q;
            load_words(rec + L::kValues + (blk * 16 + n) * (D / 8) + 8 * g, r.v[i][b]);
            load_words(rec + L::kValuePairs + (blk * L::kGroups + g) * 16, r.vp[i][b]);
        }
    }
}

__device__ __forceinline__ h8 join_scaled(const h2 (&c)[4], h2 step, h2 mid) {
    return join(__builtin_elementwise_fma(c[0], step, mid), __builtin_elementwise_fma(c[1], step, mid),
                __builtin_elementwise_fma(c[2], step, mid), __builtin_elementwise_fma(c[3], step, mid));
}

template <int D, bool BF16>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void attn4_prompt_kernel(const Attn4Args a) {
    using L = Kv4Page<D>;
    constexpr int NG = L::kGroups, NS = L::kSteps, NT = BF16 ? 1 : 2;
    constexpr int RT = Prompt<D, BF16>::kRt, ROWS = Prompt<D, BF16>::kRows;
    __shared__ h8 kfrag[2][4 * NS * 64], vfrag[2][8 * NG * 64];
    __shared__ __align__(16) uint32_t pairs[2][BF16 ? 4 : 2 * D];   // fp32 calls: 8 D bytes a page
    __shared__ uint32_t smax_all[2][4], ones[2];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, quad = lane >> 4;
    const uint32_t G = (uint32_t)a.heads / (uint32_t)a.c.kv_heads;
    // heads first: with eight of them a head's tiles share an XCD and its L2;
    // the last tiles, which see the most of a prompt, before the first
    const uint32_t x = blockIdx.x / (uint32_t)a.c.kv_heads;
    const int kv_head = (int)(blockIdx.x - x * a.c.kv_heads);
    const uint32_t tile = x / (uint32_t)a.splits;
    const int split = (int)(x - tile * a.splits);
    const uint32_t tiles = gridDim.x / ((uint32_t)a.c.kv_heads * (uint32_t)a.splits);
    const Tile t = find_tile<ROWS>(a, tiles - 1 - tile, G);
    if (t.rows == 0) return;   // the whole workgroup
    const int i_begin = min(split * a.chunk, t.pages);
    const int i_end = split == a.splits - 1 ? t.pages : min(i_begin + a.chunk, t.pages);

    // ---- this lane's rows and their queries
    uint32_t row[RT];
    int pos[RT], low[RT];
    h8 qf[RT][NT][NS], cf[RT];
    float qs[RT];
    const uint32_t wave_row = t.row0 + wave * 16 * RT;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        row[rt] = min(wave_row + 16 * rt + n, t.rows - 1);
        const uint32_t tok = row[rt] / G;
        pos[rt] = t.pos0 + (int)tok;
        low[rt] = a.window > 0 ? pos[rt] - a.window + 1 : 0;
        load_query<D, BF16, false>(a, t.token0 + (int)tok, kv_head * (int)G + (int)(row[rt] - tok * G),
                                   quad, qf[rt], cf[rt], qs[rt]);
    }
    // the wave's first and last row
    const int pos_first = t.pos0 + (int)(min(wave_row, t.rows - 1) / G);
    const int pos_last = t.pos0 + (int)(min(wave_row + 16 * RT, t.rows) - 1) / (int)G;
    const int low_last = a.window > 0 ? pos_last - a.window + 1 : 0;
    const bool idle = wave_row >= t.rows;

    const int32_t *table = a.c.table + (int64_t)t.seq * a.c.max_pages;
    auto page_at = [&](int i) { return i < t.sink_pages ? i : t.first + i - t.sink_pages; };
    const uint8_t *cache = a.c.cache + (int64_t)kv_head * L::kBytes;
    const int64_t page_bytes = (int64_t)a.c.kv_heads * L::kBytes;
    // the next page that is there, in every wave the same: 64 table entries at a
    // time, one a lane
    int from = i_begin - 64, ids = -1, id = 0;
    uint64_t there = 0;
    auto next = [&]() {
        while (there == 0) {
            from += 64;
            if (from >= i_end) {
                from = i_end;
                return -1;
            }
            const int mine = from + lane;
            ids = mine < i_end ? table[page_at(mine)] : -1;
            there = __ballot(ids >= 0 && ids < a.c.n_pages);
        }
        const int j = __builtin_ctzll(there);
        there &= there - 1;
        id = __builtin_amdgcn_readlane(ids, j);
        return page_at(from + j) * kPage;
    };
    RawQuarter<D> raw;
    uint32_t raw_pairs[D / 128 ? D / 128 : 1];   // fp32 calls: this thread's words of the pairs
    auto load = [&]() {
        const uint8_t *rec = cache + id * page_bytes;
        load_quarter<D>(rec, lane, wave, raw);
        if constexpr (!BF16) {
            const uint32_t *w = reinterpret_cast<const uint32_t *>(rec + L::kKeyPairs);
#pragma unroll
            for (int i = 0; i < (D + 127) / 128; ++i)
                raw_pairs[i] = w[(threadIdx.x + 256 * i) % (2 * D)];
        }
    };
    const uint32_t one = ones_1024();
    // fragments of the loaded page, whose first token is t0, into buffer `to`
    auto stage = [&](int t0, int to) {
        const int left = t.held - t0;   // tokens behind these have pairs of any value
#pragma unroll
        for (int j = 0; j < NS; ++j) {
            h2 c[4];
            codes8<false>(raw.k[j], one, c);
            const h2 p = as_h2(raw.kp[j >> 1]);
            kfrag[to][(wave * NS + j) * 64 + lane] =
                BF16 ? join_scaled(c, h2{p[0], p[0]}, h2{p[1], p[1]})
                     : join(c[0], c[1], c[2], c[3]);
        }
#pragma unroll
        for (int i = 0; i < RawQuarter<D>::kUnits; ++i) {
            const int u = wave + 4 * i;
            if (u >= 2 * NG) continue;
            const int hf = u / NG, g = u % NG;
            h2 c[4][4];   // [two tokens][channel]
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                codes8<false>(raw.v[i][w >> 1][w & 1], one, c[w]);
                if constexpr (BF16) {
                    uint32_t st = raw.vp[i][w >> 1][w & 1], md = raw.vp[i][w >> 1][2 + (w & 1)];
                    const int tok = 16 * (2 * hf + (w >> 1)) + 4 * quad + 2 * (w & 1);
                    const uint32_t keep = tok + 1 < left ? 0xffffffffu : tok < left ? 0xffffu : 0u;
                    st &= keep;
                    md &= keep;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        c[w][e] = __builtin_elementwise_fma(c[w][e], as_h2(st), as_h2(md));
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
                vfrag[to][((hf * NG + g) * 4 + e) * 64 + lane] =
                    join(c[0][e], c[1][e], c[2][e], c[3][e]);
        }
        if constexpr (!BF16) {
            uint32_t smax = 0;
#pragma unroll
            for (int i = 0; i < (D + 127) / 128; ++i) {
                const int w = threadIdx.x + 256 * i;
                if (w >= 2 * D) continue;
                uint32_t v = raw_pairs[i];
                if (w >= D) {   // value pairs: halfword h is of token 4 (h / 8 / NG) + h % 4
                    const int h = 2 * (w - D), tok = 4 * (h / (8 * NG)) + (h & 3);
                    v &= tok + 1 < left ? 0xffffffffu : tok < left ? 0xffffu : 0u;
                    if (!(w & 2)) smax = max(smax, max(v & 0xffffu, v >> 16));
                }
                pairs[to][w] = v;
            }
            const int top = wave_max_u16((int)smax);
            if (lane == 0) smax_all[to][wave] = (uint32_t)top;
        }
    };

    // What is carried along the pages, as in attn4_kernel, for each of the lane's
    // rows; the weights are 2^(x - m + 7), where m may stay up to 8 behind the
    // largest x, so that the accumulators are rescaled seldom.
    constexpr float kBehind = 8.0f, kUp = 7.0f;
    float m[RT];
    int E = -14;
    f4 o[RT][NG][4], sums[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        m[rt] = kNoMax;
        sums[rt] = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[rt][g][i] = f4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    if (threadIdx.x < 2) ones[threadIdx.x] = 0x3c003c00u;

    auto scores = [&](int t0, int buf, float (&s)[RT][4][4]) {
#pragma unroll
        for (int i4 = 0; i4 < 4; ++i4) {
            f4 acc[RT][BF16 ? 1 : NG];
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int g = 0; g < (BF16 ? 1 : NG); ++g) acc[rt][g] = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int j = 0; j < NS; ++j) {
                const h8 kf = kfrag[buf][(i4 * NS + j) * 64 + lane];
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int n2 = 0; n2 < NT; ++n2) {
                        f4 &c = acc[rt][BF16 ? 0 : j >> 1];
                        c = mfma(kf, qf[rt][n2][j], c);
                    }
            }
            if constexpr (BF16) {
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[rt][i4][e] = acc[rt][0][e];
            } else {
                h8 pf = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const h2 p = as_h2(pairs[buf][(16 * i4 + n) * NG + g]);
                    pf[2 * g] = p[0];
                    pf[2 * g + 1] = p[1];
                }
                const uint32_t *kp = &pairs[buf][(16 * i4 + 4 * quad) * NG];
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    const f4 rest = mfma(pf, cf[rt], f4{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        s[rt][i4][e] = rest[e] * 0x1p11f;
#pragma unroll
                        for (int g = 0; g < NG; ++g)
                            s[rt][i4][e] = fmaf((float)as_h2(kp[e * NG + g])[0], acc[rt][g][e],
                                                s[rt][i4][e]);
                    }
                }
            }
        }
        const bool all_seen =
            t0 + kPage - 1 <= pos_first && (t0 >= low_last || t0 + kPage <= a.sinks);
        if (!all_seen) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int i4 = 0; i4 < 4; ++i4)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = t0 + 16 * i4 + 4 * quad + e;
                        const bool hidden = (j > pos[rt]) | ((j < low[rt]) & (j >= a.sinks));
                        s[rt][i4][e] = hidden ? -INFINITY : s[rt][i4][e];
                    }
        }
    };
    auto weigh = [&](int buf, float (&s)[RT][4][4]) {
        int E_new = E;
        if constexpr (!BF16) {
            const uint32_t top = max(max(smax_all[buf][0], smax_all[buf][1]),
                                     max(smax_all[buf][2], smax_all[buf][3]));
            E_new = max(E, (__builtin_amdgcn_readfirstlane((int)top) >> 10) - 14);
        }
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            float top = -INFINITY;
#pragma unroll
            for (int i4 = 0; i4 < 4; ++i4)
#pragma unroll
                for (int e = 0; e < 4; ++e) top = fmaxf(top, s[rt][i4][e]);
            top = quad_max(top) * qs[rt];
            if (E_new > E || __any(top > m[rt] + kBehind)) {
                const float m_new = fmaxf(m[rt], top);
                const float f = __builtin_amdgcn_exp2f(m[rt] - m_new), fs = ldexpf(f, E - E_new);
                sums[rt] *= f;
#pragma unroll
                for (int g = 0; g < NG; ++g)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[rt][g][i] *= fs;
                m[rt] = m_new;
            }
            const float ref = m[rt] - kUp;
#pragma unroll
            for (int i4 = 0; i4 < 4; ++i4)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    s[rt][i4][e] = __builtin_amdgcn_exp2f(fmaf(s[rt][i4][e], qs[rt], -ref));
        }
        E = E_new;
        const _Float16 down = BF16 ? (_Float16)1.0f : pow2_f16(-E);
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            h2 p[RT][NT][4];
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const float p0 = s[rt][2 * hf + (w >> 1)][2 * (w & 1)];
                    const float p1 = s[rt][2 * hf + (w >> 1)][2 * (w & 1) + 1];
                    p[rt][0][w] = h2{(_Float16)p0, (_Float16)p1};
                    if constexpr (NT == 2)
                        p[rt][NT - 1][w] = h2{(_Float16)(p0 - (float)p[rt][0][w][0]),
                                              (_Float16)(p1 - (float)p[rt][0][w][1])};
                }
            h2 from4[4];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const uint32_t *src =
                    BF16 || n == 2 * NG + 1
                        ? ones
                        : &pairs[buf][D + (4 * (2 * hf + (w >> 1)) + quad) * NG * 4 +
                                      2 * (n & (2 * NG - 1))];
                from4[w] = as_h2(src[w & 1]);
            }
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int n2 = 0; n2 < NT; ++n2)
                    sums[rt] = mfma(join(from4[0], from4[1], from4[2], from4[3]),
                                    join(p[rt][n2][0], p[rt][n2][1], p[rt][n2][2], p[rt][n2][3]),
                                    sums[rt]);
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                h2 ps[RT][NT][4];
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    if constexpr (BF16) {
#pragma unroll
                        for (int rt = 0; rt < RT; ++rt) ps[rt][0][w] = p[rt][0][w];
                    } else {
                        const h2 st = as_h2(pairs[buf][D + ((4 * (2 * hf + (w >> 1)) + quad) * NG + g) * 4 +
                                                       (w & 1)]) * down;
#pragma unroll
                        for (int rt = 0; rt < RT; ++rt) {
                            ps[rt][0][w] = p[rt][0][w] * st;
                            ps[rt][NT - 1][w] = __builtin_elementwise_fma(
                                p[rt][NT - 1][w], st,
                                __builtin_elementwise_fma(p[rt][0][w], st, -ps[rt][0][w]));
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const h8 vf = vfrag[buf][((hf * NG + g) * 4 + i) * 64 + lane];
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                        for (int n2 = 0; n2 < NT; ++n2)
                            o[rt][g][i] = mfma(vf,
                                               join(ps[rt][n2][0], ps[rt][n2][1], ps[rt][n2][2],
                                                    ps[rt][n2][3]),
                                               o[rt][g][i]);
                }
            }
        }
    };

    // one page in LDS being worked on, the next one in registers or on its way
    int t0 = next(), t1 = -1;
    if (t0 >= 0) {
        load();
        stage(t0, 0);
        t1 = next();
        if (t1 >= 0) load();
    }
    for (int buf = 0; t0 >= 0; buf ^= 1) {
        __syncthreads();   // the page is whole, and everyone is done with the other buffer
        const bool seen = !idle && t0 <= pos_last;
        float s[RT][4][4];
        if (seen) scores(t0, buf, s);
        int t2 = -1;
        if (t1 >= 0) {
            stage(t1, buf ^ 1);
            t2 = next();
            if (t2 >= 0) load();
        }
        if (seen) weigh(buf, s);
        t0 = t1;
        t1 = t2;
    }

    // ---- everything of a row is scaled by 2^(kUp - m)
    const float up = ldexpf(1.0f, E);
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        constexpr int kOnes = BF16 ? 0 : 2 * NG + 1;
        const float l = __shfl(sums[rt][kOnes & 3], n + 16 * (kOnes >> 2));
        const bool mine = wave_row + 16 * rt + n < t.rows;
        const uint32_t tok = row[rt] / G;
        const int64_t line =
            (int64_t)(t.token0 + (int)tok) * a.heads + kv_head * G + (row[rt] - tok * G);
        float *part = a.part + ((int64_t)split * a.N * a.heads + line) * (D + 4);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const float rest =
                BF16 ? 0.0f : __shfl(sums[rt][(2 * g + 1) & 3], n + 16 * ((2 * g + 1) >> 2));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int ch = 64 * g + 16 * quad + 4 * e;
                float4 w;
                w.x = BF16 ? o[rt][g][0][e] : fmaf(o[rt][g][0][e], up, rest);
                w.y = BF16 ? o[rt][g][1][e] : fmaf(o[rt][g][1][e], up, rest);
                w.z = BF16 ? o[rt][g][2][e] : fmaf(o[rt][g][2][e], up, rest);
                w.w = BF16 ? o[rt][g][3][e] : fmaf(o[rt][g][3][e], up, rest);
                if (!mine) continue;
                if (a.splits > 1) *reinterpret_cast<float4 *>(part + ch) = w;
                else store_out<BF16>(a.out, line * D + ch, w, l);
            }
        }
        if (mine && a.splits > 1 && quad == 0) {
            part[D] = m[rt];
            part[D + 1] = l;
        }
    }
}

// Joins the splits of a row: D / 4 lanes to its channels, `par` (a power of
// two) groups of them to its splits, always added in the same order.  A part
// without a sum has no accumulators.
template <int D, bool BF16>
__global__ __launch_bounds__(kJoinThreads) void attn4_join_kernel(const Attn4Args a, int par) {
    constexpr int kLanes = D / 4, kMaxSlots = kJoinThreads / kLanes;
    __shared__ float4 o_all[kJoinThreads];
    __shared__ float m_all[kMaxSlots], l_all[kMaxSlots];
    const int slots = blockDim.x / kLanes;
    const int slot = threadIdx.x / kLanes, ch = 4 * (threadIdx.x % kLanes);
    const int g = slot & (par - 1);
    const int64_t line = (int64_t)blockIdx.x * (slots / par) + slot / par, lines = a.N * a.heads;
    const bool mine = line < lines && row_in_call(a.c, line / a.heads);
    const float *part = a.part + line * (D + 4);
    const int64_t stride = lines * (D + 4);
    float top = kNoMax, sum = 0.0f;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (mine) {
        // four parts at a time, all of their loads before the first use
        constexpr int kBatch = 4;
        for (int s = g; s < a.splits; s += kBatch * par) {
            float ms[kBatch], ls[kBatch], best = top;
            float4 os[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const float *p = part + min(s + i * par, a.splits - 1) * stride;
                os[i] = *reinterpret_cast<const float4 *>(p + ch);
                ms[i] = p[D];
                ls[i] = p[D + 1];
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                if (s + i * par >= a.splits) ls[i] = 0.0f;
                if (ls[i] > 0.0f) best = fmaxf(best, ms[i]);
                else os[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
            const float f = __builtin_amdgcn_exp2f(top - best);
            sum *= f;
            acc.x *= f; acc.y *= f; acc.z *= f; acc.w *= f;
            top = best;
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                add_part(acc, sum, ls[i] > 0.0f ? __builtin_amdgcn_exp2f(ms[i] - top) : 0.0f,
                         os[i], ls[i]);
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
    const int rows = a.prompt ? Prompt<D, BF16>::kRows : kRows;
    const int64_t tiles = a.N * G / rows + a.c.n_seqs;
    const dim3 grid((unsigned)(tiles * a.c.kv_heads * a.splits));
    if (a.prompt)
        hipLaunchKernelGGL((attn4_prompt_kernel<D, BF16>), grid, dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL((attn4_kernel<D, BF16>), grid, dim3(64 * kWaves), 0, st, a);
    if (a.splits > 1) {
        // few rows with many splits: whole workgroups of 1024 to a row
        const int64_t lines = a.N * a.heads;
        const int threads = a.splits > 16 ? kJoinThreads : 256, slots = threads / (D / 4);
        int par = 1;
        while (par < slots && 2 * par < a.splits) par *= 2;
        const int64_t per = slots / par;
        hipLaunchKernelGGL((attn4_join_kernel<D, BF16>),
                           dim3((unsigned)((lines + per - 1) / per)), dim3(threads), 0, st, a, par);
    }
}

}  // namespace

Attn4Plan attn4_plan(int64_t n_seqs, int64_t N, int64_t heads, int64_t kv_heads, int64_t max_kv,
                     int64_t window, int64_t sinks) {
    // Prompts go where a sequence has kPromptFrom rows on average.  Chunks of
    // pages, so that a batch's workgroups are alike however its lengths differ:
    // enough of them for kWanted workgroups, each at least one page for every wave
    // (prompts: kPromptChunk pages, since a workgroup has its rows to prepare).
    const int64_t rows = N * (heads / kv_heads);
    const bool prompt = rows >= kPromptFrom * n_seqs;
    const int64_t tile = prompt ? 128 : kRows, least = prompt ? kPromptChunk : kWaves;
    const int64_t groups = (rows / tile + n_seqs) * kv_heads;
    int64_t pages = (max_kv + kPage - 1) / kPage;
    if (window > 0)   // what a tile's rows can see of it: the window before each, the sinks
        pages = std::min(pages, (window + tile) / kPage + 2 + (sinks + kPage - 1) / kPage);
    int64_t s = (kWanted + groups - 1) / groups;
    if (s > kMaxSplits) s = kMaxSplits;
    int64_t chunk = (pages + s - 1) / s;
    chunk = chunk < least ? least : (chunk + kWaves - 1) / kWaves * kWaves;
    s = (pages + chunk - 1) / chunk;
    return Attn4Plan{prompt ? 1 : 0, s < 1 ? 1 : (int)s, (int)chunk};
}

hipError_t launch_attn4(const Attn4Args &a, int bf16, int dim, hipStream_t st) {
    if (dim == 64) { if (bf16) launch_d<64, true>(a, st); else launch_d<64, false>(a, st); }
    else if (dim == 128) { if (bf16) launch_d<128, true>(a, st); else launch_d<128, false>(a, st); }
    else { if (bf16) launch_d<256, true>(a, st); else launch_d<256, false>(a, st); }
    return hipGetLastError();
}

}  // namespace bitnet
