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
// q is scaled by a power of two per row, the steps by one that goes by the page, which
// is visited again where its steps span too much for one, so both are normal numbers
// in fp16; bf16 calls round p and p * step once to fp16's 11 bits, finer than the
// output (q's 8 are exact), fp32 calls carry them and q as two fp16 terms (22 bits).
// Both end at 2^-25, far below a row's largest weight (kUp).  Sums, maxima and
// accumulators are fp32.
//
// The first product is taken transposed (tokens x rows), which leaves a lane
// with 16 tokens of one row: that is exactly the fragment that the second
// product (channels x rows) takes, so p never crosses lanes, and the running
// maximum and the accumulators of a row all live in the same lanes.
//
// What bounds it.  A long history of few rows: HBM with bf16 rows (64 sequences of
// up to 4096 tokens, 64/8 heads of 128: 175 MB in 36 to 41 us, the less of it the
// last-level cache holds the more; a large copy reaches 4.8 TB/s), the vector
// operations with fp32 rows (131072 tokens, 20/5 heads: 94 MB in 26 us, and 5 us for
// the join; the batch of 64 in 61 us): a page of 128 channels costs a wave about 600
// of them (350 in bf16 calls) and 72 (38) matrix instructions, however many of its 16
// rows are real; the unpacking is the largest part.  Prompts: the vector operations
// again, of which 32 rows a wave share the unpacking (three of 2048 tokens, 16/8
// heads of 128, bf16: 36 GF in 72 us, 500 TF; they fill 71% of the cycles of a busy
// compute unit, the matrix instructions 29%).  Short histories: the chain of dependent
// loads (lengths, table, page), a page or two of work and the join of the
// waves (515 tokens, 20/5 heads, fp32: 9.6 us in a graph).
#include <algorithm>

#include "kv4.h"

namespace bitnet {

namespace {

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef uint16_t us2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));

constexpr int kJoinThreads = 1024;
constexpr float kNoMax = -3.0e38f; // a running maximum before the first visible token

__device__ __forceinline__ us2 as_us2(uint32_t w) { return __builtin_bit_cast(us2, w); }
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
// The steps in a word of two that are below `cut`; the others 0.
__device__ __forceinline__ uint32_t steps_below(uint32_t w, uint32_t cut) {
    return ((w & 0xffffu) < cut ? w & 0xffffu : 0) | (w >> 16 < cut ? w & 0xffff0000u : 0);
}
// 2^e as fp16 (0 where that has none so small), e <= 16.
__device__ __forceinline__ uint32_t half_bits(int e) {
    return e >= -14 ? (e + 15) << 10 : e >= -24 ? 1 << (e + 24) : 0;
}
__device__ __forceinline__ _Float16 pow2_f16(int e) {
    return __builtin_bit_cast(_Float16, (uint16_t)half_bits(e));
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
    // a sequence has at least as many tiles to itself as its rows need
    const SeqAt s = sequence_of<ROWS, 1>(a.c, G, x);
    t.seq = s.seq;
    t.token0 = s.begin;
    const bool good = s.begin >= 0 && s.end > s.begin && s.end <= (int)a.N;
    t.rows = good ? (uint32_t)(s.end - s.begin) * G : 0;
    const int tile = (int)(x - ((uint32_t)s.begin * G / ROWS + s.seq));
    if (tile < 0) t.rows = 0;
    t.row0 = (uint32_t)tile * ROWS;
    t.held = s.held;
    t.pos0 = t.held - (s.end - s.begin);
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

__device__ __forceinline__ void add_part(float4 &acc, float f, const float4 &o) {
    acc.x = fmaf(f, o.x, acc.x);
    acc.y = fmaf(f, o.y, acc.y);
    acc.z = fmaf(f, o.z, acc.z);
    acc.w = fmaf(f, o.w, acc.w);
}
// Four channels of a finished row; inv: one over its sum, or 0 if it saw nothing.
template <bool BF16>
__device__ __forceinline__ void store_out(void *out, int64_t at, float4 acc, float inv) {
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

// The pages [begin, end) of a tile's list that a split takes: shares of what this
// tile's rows see, so a call captured for the longest history loses little on a
// short one (8 sequences, 32/8 heads of 128, bf16, captured for 32768 tokens: at 4000
// 14.3 us, as if captured for 4000, against 34.6 with shares of the longest; two pages
// to a wave are not split, 8.9 against 11.0 us at 500).  A tile whose pages are one split's has its result written by it; its
// part then says so in place of a sum, and the join leaves the row alone.
constexpr float kFinal = -1.0f;
struct Share {
    int begin, end;
    bool shared;
};
__device__ __forceinline__ Share share_of(const Attn4Args &a, const Tile &t, int split) {
    const bool whole = a.splits == 1 || (a.splits > 2 && t.pages <= 8);
    const int chunk = whole ? t.pages : chunk_of(t.pages, a.splits);
    Share s;
    s.begin = min(split * chunk, t.pages);
    s.end = min(s.begin + chunk, t.pages);
    s.shared = t.pages > chunk;
    return s;
}
// The output line of a sequence's row r, and its part of a split.
__device__ __forceinline__ int64_t line_of(const Attn4Args &a, const Tile &t, uint32_t r, int kv_head,
                                           uint32_t G) {
    const uint32_t tok = r / G;
    return (int64_t)(t.token0 + (int)tok) * a.heads + kv_head * (int)G + (int)(r - tok * G);
}
template <int D>
__device__ __forceinline__ float *part_of(const Attn4Args &a, int split, int64_t line) {
    return a.part + ((int64_t)split * a.N * a.heads + line) * (D + 4);
}
// A split without pages leaves parts without a sum, where they are looked at.
template <int D>
__device__ __forceinline__ void write_nothing(const Attn4Args &a, const Tile &t, const Share &s,
                                              int kv_head, uint32_t G, int split, uint32_t rows) {
    const uint32_t lane = threadIdx.x & 63, r = t.row0 + lane;
    if (s.shared && lane < rows && r < t.rows)
        part_of<D>(a, split, line_of(a, t, r, kv_head, G))[D + 1] = 0.0f;
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
    // q times 2^k: the largest is in [2^14, 2^15) (a row of numbers below 2^-111
    // stays smaller).  The sums of q: with raw codes times 2^(k - 24), the product's
    // own scale (to 2^-25, 2^-16 of the largest q); else times 2^(k - 11), the
    // largest they can be being 2^10, and scaled after their product.
    const int k = top > 0.0f ? min(15 - __builtin_amdgcn_frexp_expf(top), 126) : 0;
    const float up = ldexpf(1.0f, k), up16 = up * 0.0625f;
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
                const float z = v[j][ch] * (RAW && (e & 2) ? up16 : up);
                const _Float16 hi = (_Float16)z;
                qf[0][j][e] = hi;
                if constexpr (!BF16) qf[1][j][e] = (_Float16)(z - (float)hi);
                sum = fmaf(v[j][ch], up * (RAW ? 0x1p-24f : 0x1p-11f), sum);
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

// A tile has 16 * RT rows, 16 to each of RT fragments; TURNS waves take turns at
// its pages, and a workgroup has WAVES / TURNS tiles.  RT is 2 for prompts of many
// rows, which shares what a page's codes cost to unpack; eight waves serve a single
// short history, which is then not split.
constexpr int least_waves(int dim, int rt, int waves) {   // to a SIMD
    return waves == 4 && dim * rt <= 128 ? 3 : 2;
}
// Whether a tile's query lies in LDS (where the waves' results meet later) instead
// of registers, so that a SIMD holds that many waves without spills: rows of 256
// channels 2 in place of 1 (two prompts of 2048, 16/4 heads, bf16: 185 -> 110 us),
// fp32 rows of 128 3 in place of 2 (one of 512, 20/5 heads: 18 -> 14 us).  fp32 rows
// of 64 in two fragments spill a few registers for their third wave and gain by it
// (four prompts of 2048, 32/8 heads: 200 -> 182 us), as much as from LDS.
constexpr bool query_in_lds(int dim, bool bf16, int waves) {
    return dim == 256 || (dim == 128 && !bf16 && waves == 4);
}

template <int D, bool BF16, int RT, int WAVES, int TURNS>
__global__ __launch_bounds__(64 * WAVES, least_waves(D, RT, WAVES)) void attn4_kernel(
    const Attn4Args a) {
    using L = Kv4Page<D>;
    constexpr int NG = L::kGroups, NS = L::kSteps, NT = BF16 ? 1 : 2, ROWS = 16 * RT;
    // The weights p are 2^(x - m + kUp), where m may stay up to kBehind behind the largest
    // x so that the accumulators are rescaled seldom.  What fp16 holds of p ends at 2^-25,
    // so a token's part is off by up to 2^-(25 + kUp) of its value at the largest weight:
    // 2^-37 with fp32 rows, 2^-32 with bf16.  (7 bits for fp32 rows too would cost up to
    // 1.5% less, but 2^-32 of a value of 20000 next to one of 0.01 is 2^-11 of that.)
    constexpr float kUp = BF16 ? 7.0f : 12.0f, kBehind = 15.0f - kUp;
    constexpr int SUBS = 2;   // 16-token quarters of a page that are worked on together
    constexpr int kCodeExp = BF16 ? 24 : 0;   // raw codes carry 2^-24, and every second pair 16
    __shared__ __align__(16) uint32_t pairs_all[WAVES][2 * D];   // 8 D bytes a page
    __shared__ __align__(16) uint32_t ones_all[WAVES][2];        // four fp16 ones
    __shared__ __align__(16) float4 o_all[WAVES][RT * NG * 4][64];
    __shared__ float m_all[WAVES][ROWS], l_all[WAVES][ROWS];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, quad = lane >> 4;
    uint32_t *const pairs = pairs_all[wave], *const ones = ones_all[wave];
    const uint32_t G = (uint32_t)a.heads / (uint32_t)a.c.kv_heads;
    // heads first: with eight of them a head's tiles share an XCD and its L2;
    // a prompt's last tiles, which see the most, before its first
    const uint32_t x = blockIdx.x / (uint32_t)a.c.kv_heads;
    const int kv_head = (int)(blockIdx.x - x * a.c.kv_heads);
    const uint32_t tile = x / (uint32_t)a.splits;
    const int split = (int)(x - tile * a.splits);
    constexpr int TEAMS = WAVES / TURNS;
    // the waves that have a page more than the others are not the same of all splits
    const int team = wave / TURNS, turn = (wave + split) % TURNS;
    Tile t = find_tile<ROWS>(a, a.tiles - 1 - (tile * TEAMS + team), G);
    Share sh = share_of(a, t, split);
    if constexpr (TEAMS == 1) {   // the whole workgroup leaves
        if (t.rows == 0) return;
        if (sh.begin == sh.end && split > 0) {
            if (turn == 0) write_nothing<D>(a, t, sh, kv_head, G, split, ROWS);
            return;
        }
    } else if (t.rows == 0) {   // a team without rows stays for the barrier
        t.token0 = 0;
        t.row0 = 0;
        sh = Share{0, 0, false};
    }
    const uint32_t last_row = t.rows > 0 ? t.rows - 1 : 0;

    // ---- the pages of this split, every TURNS-th to this wave.  64 table entries
    // at a time, one a lane, with a bit for each page that is there; they are
    // waited for before the pages, so that no wait of the loop takes in a page that
    // is on its way.  For the same reason a page is always loaded, at the end the
    // last one again (from the L2): the count of loads in flight is then the same
    // on every path.
    const int32_t *table = a.c.table + (int64_t)t.seq * a.c.max_pages;
    auto page_at = [&](int i) { return i < t.sink_pages ? i : t.first + i - t.sink_pages; };
    const uint8_t *cache = a.c.cache + (int64_t)kv_head * L::kBytes;
    const int64_t page_bytes = (int64_t)a.c.kv_heads * L::kBytes;
    int from = sh.begin + turn, ids = -1, id = 0, at_bit = 0;
    uint64_t there = 0;
    auto load_ids = [&]() {
        const int mine = from + TURNS * lane;
        ids = mine < sh.end ? table[page_at(mine)] : -1;
        there = __ballot(ids >= 0 && ids < a.c.n_pages);
    };
    // the next page: its first token, or -1; its record is at `rec`
    const uint8_t *rec = cache;
    auto next = [&]() {
        while (there == 0) {
            if (from >= sh.end - 64 * TURNS) return -1;
            from += 64 * TURNS;
            load_ids();
        }
        at_bit = __builtin_ctzll(there);
        there &= there - 1;
        id = __builtin_amdgcn_readlane(ids, at_bit);
        rec = cache + id * page_bytes;
        return page_at(from + TURNS * at_bit) * kPage;
    };
    // codes of the quarters that come next, and this lane's share of a page's pairs
    uint32_t raw_k[SUBS][D / 32], raw_v[SUBS][D / 32], raw_m[D / 32];
    auto load_keys = [&](const uint8_t *r, int sub) {
#pragma unroll
        for (int i = 0; i < SUBS; ++i)
            load_words(r + (16 * (sub + i) + n) * L::kRow + quad * (D / 8), raw_k[i]);
    };
    auto load_pairs = [&](const uint8_t *r) {
        load_words(r + L::kKeyPairs + lane * (D / 8), raw_m);
    };
    auto load_values = [&](const uint8_t *r, int sub) {
#pragma unroll
        for (int i = 0; i < SUBS; ++i)
            load_words(r + L::kValues + ((4 * (sub + i) + quad) * 16 + n) * (D / 8), raw_v[i]);
    };
    load_ids();
    int t0 = next();
    load_pairs(rec);
    load_keys(rec, 0);
    load_values(rec, 0);

    // ---- this lane's rows and their queries, 8 channels of every 32
    const uint32_t one = BF16 ? 0 : ones_1024();
    int pos[RT], low[RT];
    h8 qf[RT][NT][NS], cf[RT];
    float qs[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const uint32_t row = min(t.row0 + 16 * rt + n, last_row), tok = row / G;
        pos[rt] = t.pos0 + (int)tok;
        low[rt] = a.window > 0 ? pos[rt] - a.window + 1 : 0;   // may be negative
        load_query<D, BF16, BF16>(a, t.token0 + (int)tok, kv_head * (int)G + (int)(row - tok * G),
                                  quad, qf[rt], cf[rt], qs[rt]);
    }
    constexpr bool kQueryInLds = query_in_lds(D, BF16, WAVES);
    h8 *const q_lds = reinterpret_cast<h8 *>(o_all) + team * RT * NT * NS * 64 + lane;
    if constexpr (kQueryInLds) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int n2 = 0; n2 < NT; ++n2)
#pragma unroll
                for (int j = 0; j < NS; ++j)
                    if (j % TURNS == turn) q_lds[((rt * NT + n2) * NS + j) * 64] = qf[rt][n2][j];
        __syncthreads();
    }
    const int pos_first = t.pos0 + (int)(t.row0 / G);
    const int low_last = a.window > 0
                             ? t.pos0 + (int)(min(t.row0 + ROWS - 1, last_row) / G) - a.window + 1
                             : 0;
    // Tokens that may not have been written: behind the sequence's last, and those that the
    // windows of all rows hide.  Pages that begin in [seen_from, seen_from + seen) have none.
    const int seen_from = a.window > 0 ? max(pos_first - a.window + 1, 0) : 0;
    const uint32_t seen = (uint32_t)max(t.held - kPage + 1 - seen_from, 0);
    auto unseen = [&](int j) { return j >= t.held || (j < seen_from && j >= a.sinks); };

    // What is carried along the pages.  The steps in front of the second product are
    // divided by 2^E.  `sums` is the product of p with what row n of 16 stands for: row
    // 2 g the steps of group g, 2 g + 1 its middles, 2 NG + 1 ones.
    float m[RT];
    int E = 2;                   // the steps of the page are below 2^E
    const bool steps_here = lane >= 32 && (D > 64 || !(lane & 1));   // see raw_m below
    _Float16 down = steps_here ? pow2_f16(-E) : (_Float16)1.0f;      // 2^-E for the steps
    f4 o[RT][NG][4], sums[RT];   // o[..][g][i][e]: channel 64 g + 16 quad + 4 e + i
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        m[rt] = kNoMax;
        sums[rt] = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[rt][g][i] = f4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    // Pages whose steps are all in [2^(E - 10), 2^E) are taken as they are: divided by 2^E
    // they are normal numbers, and p * step is off by 2^(-15 - kUp) steps at most.  For other
    // pages E changes (where it starts suits values of about 1), and where no E does for
    // all steps of a page, those that are too small are left to another visit of it, in
    // which nothing else counts (`cut`: what they are below; E falls by nine with each
    // visit, down to -13, below which no step needs it).  As bits of fp16: `least` and
    // `span`, [least, least + span).  Zeros are looked at, and change nothing.
    auto least_of = [](int e) { return e > -13 ? half_bits(e - 10) : 0u; };
    uint32_t least = least_of(E), span = half_bits(E) - least, cut = 0;
    if (lane < 2) ones[lane] = 0x3c003c00u;
    const uint32_t *sums_from[4];   // this lane's row of `sums`, for tokens 16 i + 4 quad ..
#pragma unroll
    for (int i = 0; i < 4; ++i)
        sums_from[i] = n == 2 * NG + 1
                           ? ones
                           : &pairs[D + (4 * i + quad) * NG * 4 + 2 * (n & (2 * NG - 1))];

    while (t0 >= 0) {
        // ---- the page's pairs go through LDS, its steps divided by 2^E
        // lanes 32 on hold four steps, then four middles, and so on
        auto is_steps = [](int w) { return D == 64 || !(w & 2); };
        // what is not seen may have pairs of any value, which a weight of 0 would not silence
        auto hide = [&](uint32_t by) {
            if ((uint32_t)(t0 - seen_from) < seen || lane < 32) return;
#pragma unroll
            for (int w = 0; w < D / 32; ++w) {
                // halfword i of the value pairs: token 4 (i / 8 / NG) + i % 4
                const int h0 = (lane - 32) * (D / 16) + 2 * w;
                const int j = t0 + 4 * (h0 / (8 * NG)) + (h0 & 3);
                if (unseen(j)) raw_m[w] = (raw_m[w] & 0xffff0000u) | by;
                if (unseen(j + 1)) raw_m[w] = (raw_m[w] & 0xffffu) | by << 16;
            }
        };
        hide(least);
        us2 far = {0, 0};
#pragma unroll
        for (int w = 0; w < D / 32; ++w)
            if (is_steps(w))
                far = __builtin_elementwise_max(far, as_us2(raw_m[w]) - as_us2(least * 0x10001u));
        int E_new = E;
        if (__any(steps_here && max((uint32_t)far[0], (uint32_t)far[1]) >= span)) {
            hide(0);
            uint32_t top = 0;
            bool low = false;
#pragma unroll
            for (int w = 0; w < D / 32; ++w) {
                if (cut && lane >= 32)
                    raw_m[w] = steps_here && is_steps(w) ? steps_below(raw_m[w], cut) : 0;
                if (!steps_here || !is_steps(w)) continue;
                top = max(top, max(raw_m[w] & 0xffffu, raw_m[w] >> 16));
                low |= steps_below(raw_m[w], least) != 0;
            }
            if (lane < 2) ones[lane] = cut ? 0 : 0x3c003c00u;   // p counts once
            const int most = wave_max_u16((int)top);
            bool again = false;
            if (most >= (int)half_bits(E) || __any(low)) {
                E_new = min(most >> 10, 29) - 13;   // an octave to spare
                least = least_of(E_new);
                down = steps_here ? pow2_f16(-E_new) : (_Float16)1.0f;
                low = false;
#pragma unroll
                for (int w = 0; w < D / 32; ++w) {
                    if (!steps_here || !is_steps(w)) continue;
                    const uint32_t small = steps_below(raw_m[w], least);
                    low |= small != 0;
                    raw_m[w] ^= small;
                }
                again = __any(low);
            }
            span = cut || again ? 0 : half_bits(E_new) - least;   // 0: the next page is looked at
            cut = again ? least : 0;
            if (again) there |= (uint64_t)1 << at_bit;   // it is this one once more
        }
        {
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int w = 0; w < D / 32; ++w)
                pairs[lane * (D / 32) + w] =
                    D == 64 || !(w & 2) ? __builtin_bit_cast(uint32_t, as_h2(raw_m[w]) * down)
                                        : raw_m[w];
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        }
        const uint8_t *const rec0 = rec;
        int t1 = -1;
#pragma unroll
        for (int sub = 0; sub < 4; sub += SUBS) {
        // ---- scores: s[..][i][e] is token 16 (sub + i) + 4 quad + e
        float s[RT][SUBS][4];
#pragma unroll
        for (int i4 = 0; i4 < SUBS; ++i4) {
            h8 pf = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const h2 p = as_h2(pairs[(16 * (sub + i4) + n) * NG + g]);
                pf[2 * g] = p[0];
                pf[2 * g + 1] = p[1];
            }
            f4 acc[RT][NG];
#pragma unroll
            for (int g = 0; g < NG; ++g) {
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) acc[rt][g] = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int j = 2 * g; j < 2 * g + 2; ++j) {
                    h2 c[4];
                    codes8<BF16>(raw_k[i4][j], one, c);
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                        for (int n2 = 0; n2 < NT; ++n2)
                            acc[rt][g] =
                                mfma(join(c[0], c[1], c[2], c[3]),
                                     kQueryInLds ? q_lds[((rt * NT + n2) * NS + j) * 64] : qf[rt][n2][j],
                                     acc[rt][g]);
                }
            }
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                const f4 rest = mfma(pf, cf[rt], f4{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[rt][i4][e] = BF16 ? rest[e] : rest[e] * 0x1p11f;
#pragma unroll
                    for (int g = 0; g < NG; ++g)
                        s[rt][i4][e] =
                            fmaf((float)as_h2(pairs[(16 * (sub + i4) + 4 * quad + e) * NG + g])[0],
                                 acc[rt][g][e], s[rt][i4][e]);
                }
            }
        }
        // the next keys come while these values are worked on, the next values
        // while the next keys are
        if (sub + SUBS < 4) {
            load_keys(rec0, sub + SUBS);
        } else {
            t1 = next();
            load_pairs(rec);
            load_keys(rec, 0);
        }
        const bool all_seen =
            t0 + kPage - 1 <= pos_first && (t0 >= low_last || t0 + kPage <= a.sinks);
        if (!all_seen) {
            asm volatile("");   // a branch: most pages are seen by all rows
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int i4 = 0; i4 < SUBS; ++i4)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = t0 + 16 * (sub + i4) + 4 * quad + e;
                        const bool hidden = (j > pos[rt]) | ((j < low[rt]) & (j >= a.sinks));
                        s[rt][i4][e] = hidden ? -INFINITY : s[rt][i4][e];
                    }
        }
        // ---- p
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            float top = -INFINITY;   // of this lane's tokens: the row's only where it matters
#pragma unroll
            for (int i4 = 0; i4 < SUBS; ++i4)
#pragma unroll
                for (int e = 0; e < 4; ++e) top = fmaxf(top, s[rt][i4][e]);
            if (E_new != E || __any(top * qs[rt] > m[rt] + kBehind)) {
                const float m_new = fmaxf(m[rt], quad_max(top) * qs[rt]);
                const float f = __builtin_amdgcn_exp2f(m[rt] - m_new), fs = ldexpf(f, E - E_new);
                sums[rt][0] *= fs;
                sums[rt][1] *= f;
                sums[rt][2] *= fs;
                sums[rt][3] *= f;
#pragma unroll
                for (int g = 0; g < NG; ++g)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[rt][g][i] *= fs;
                m[rt] = m_new;
            }
            const float ref = m[rt] - kUp;
#pragma unroll
            for (int i4 = 0; i4 < SUBS; ++i4)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    s[rt][i4][e] = __builtin_amdgcn_exp2f(fmaf(s[rt][i4][e], qs[rt], -ref));
        }
        E = E_new;
        // ---- the second product
#pragma unroll
        for (int hf = 0; hf < SUBS / 2; ++hf) {
            h2 p[RT][NT][4];   // pairs of tokens: two of 16 * 2 hf on, two of 16 (2 hf + 1) on
            h2 row[4];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                row[w] = as_h2(sums_from[sub + 2 * hf + (w >> 1)][w & 1]);
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    const float p0 = s[rt][2 * hf + (w >> 1)][2 * (w & 1)];
                    const float p1 = s[rt][2 * hf + (w >> 1)][2 * (w & 1) + 1];
                    p[rt][0][w] = h2{(_Float16)p0, (_Float16)p1};
                    if constexpr (NT == 2)
                        p[rt][NT - 1][w] = h2{(_Float16)(p0 - (float)p[rt][0][w][0]),
                                              (_Float16)(p1 - (float)p[rt][0][w][1])};
                }
            }
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int n2 = 0; n2 < NT; ++n2)
                    sums[rt] = mfma(join(row[0], row[1], row[2], row[3]),
                                    join(p[rt][n2][0], p[rt][n2][1], p[rt][n2][2], p[rt][n2][3]),
                                    sums[rt]);
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                h2 ps[RT][NT][4], c[4][4];   // p * step, and the codes [two tokens][channel]
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const h2 st = as_h2(
                        pairs[D + ((4 * (sub + 2 * hf + (w >> 1)) + quad) * NG + g) * 4 + (w & 1)]);
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) {
                        ps[rt][0][w] = p[rt][0][w] * st;
                        if constexpr (NT == 2)
                            ps[rt][NT - 1][w] = __builtin_elementwise_fma(
                                p[rt][NT - 1][w], st,
                                __builtin_elementwise_fma(p[rt][0][w], st, -ps[rt][0][w]));
                    }
                    codes8<BF16>(raw_v[2 * hf + (w >> 1)][2 * g + (w & 1)], one, c[w]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                        for (int n2 = 0; n2 < NT; ++n2)
                            o[rt][g][i] = mfma(join(c[0][i], c[1][i], c[2][i], c[3][i]),
                                               join(ps[rt][n2][0], ps[rt][n2][1], ps[rt][n2][2],
                                                    ps[rt][n2][3]),
                                               o[rt][g][i]);
            }
        }
        if (sub + SUBS < 4) load_values(rec0, sub + SUBS);
        else load_values(rec, 0);
        }
        t0 = t1;
    }

    // ---- everything of a row at one scale, 2^(kUp - m)
    const float up = ldexpf(1.0f, kCodeExp + E), up1 = BF16 ? up * 0.0625f : up;
    float l[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        auto sum_row = [&](int r) { return __shfl(sums[rt][r & 3], n + 16 * (r >> 2)); };
        l[rt] = sum_row(2 * NG + 1);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            float rest = sum_row(2 * g + 1);
            if (BF16) rest -= sum_row(2 * g) * ldexpf(8.0f, E);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    o[rt][g][i][e] = fmaf(o[rt][g][i][e], i & 1 ? up1 : up, rest);
        }
    }
    if constexpr (kQueryInLds) __syncthreads();   // all queries read
    // ---- join the waves: each takes every TURNS-th four of a lane's channels
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        if (quad == 0) {
            m_all[wave][16 * rt + n] = m[rt];
            l_all[wave][16 * rt + n] = l[rt];
        }
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                o_all[wave][(rt * NG + g) * 4 + e][lane] =
                    make_float4(o[rt][g][0][e], o[rt][g][1][e], o[rt][g][2][e], o[rt][g][3][e]);
    }
    __syncthreads();
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const int rr = 16 * rt + n;
        if (t.row0 + rr >= t.rows) continue;
        const int first = team * TURNS;
        float top = m_all[first][rr], f[TURNS];
#pragma unroll
        for (int w = 1; w < TURNS; ++w) top = fmaxf(top, m_all[first + w][rr]);
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < TURNS; ++w) {
            f[w] = __builtin_amdgcn_exp2f(m_all[first + w][rr] - top);
            sum = fmaf(f[w], l_all[first + w][rr], sum);
        }
        const int64_t line = line_of(a, t, t.row0 + rr, kv_head, G);
        float *part = part_of<D>(a, split, line);
        const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
        for (int u = 0; u < (4 * NG + TURNS - 1) / TURNS; ++u) {
            const int it = turn + u * TURNS;
            if (4 * NG % TURNS != 0 && it >= 4 * NG) continue;
            float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int w = 0; w < TURNS; ++w)
                add_part(acc, f[w], o_all[first + w][rt * NG * 4 + it][lane]);
            const int ch = 64 * (it >> 2) + 16 * quad + 4 * (it & 3);
            if (sh.shared) *reinterpret_cast<float4 *>(part + ch) = acc;
            else store_out<BF16>(a.out, line * D + ch, acc, inv);
        }
        if (a.splits > 1 && turn == 0 && quad == 0) {
            part[D] = top;
            part[D + 1] = sh.shared ? sum : kFinal;
        }
    }
}

// Joins the splits of a row: D / 4 lanes to its channels, `par` (a power of
// two) groups of them to its splits, always added in the same order.  A part
// without a sum has no accumulators.  Bound by latency: 20 rows of 98 splits, 1 MB,
// take 5 us, of which a launch is about 2.
template <int D, bool BF16>
__global__ __launch_bounds__(kJoinThreads) void attn4_join_kernel(const Attn4Args a, int par) {
    constexpr int kLanes = D / 4, kMaxSlots = kJoinThreads / kLanes;
    __shared__ float4 o_all[kJoinThreads];
    __shared__ float m_all[kMaxSlots], l_all[kMaxSlots];
    const int slots = blockDim.x / kLanes;
    const int slot = threadIdx.x / kLanes, ch = 4 * (threadIdx.x % kLanes);
    const int g = slot & (par - 1);
    const int64_t line = (int64_t)blockIdx.x * (slots / par) + slot / par, lines = a.N * a.heads;
    const float *part = a.part + line * (D + 4);
    const bool mine = line < lines && row_in_call(a.c, line / a.heads) && part[D + 1] != kFinal;
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
                // a sum that is no number goes on into the row, as without splits
                if (ls[i] != 0.0f) best = fmaxf(best, ms[i]);
                else os[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
            const float f = __builtin_amdgcn_exp2f(top - best);
            sum *= f;
            acc.x *= f; acc.y *= f; acc.z *= f; acc.w *= f;
            top = best;
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const float fi = ls[i] != 0.0f ? __builtin_amdgcn_exp2f(ms[i] - top) : 0.0f;
                sum = fmaf(fi, ls[i], sum);
                add_part(acc, fi, os[i]);
            }
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
        for (int i = 0; i < par; ++i) {
            const float fi = __builtin_amdgcn_exp2f(m_all[slot + i] - top);
            sum = fmaf(fi, l_all[slot + i], sum);
            add_part(acc, fi, o_all[threadIdx.x + i * kLanes]);
        }
    }
    if (mine) store_out<BF16>(a.out, line * D + ch, acc, sum > 0.0f ? 1.0f / sum : 0.0f);
}

// LDS that leaves `per_cu` workgroups of four waves to a compute unit (0: as many as fit).
template <int D>
int spare_lds(int per_cu) {
    constexpr int kLds = 160 * 1024, kOwn = 4 * (8 * D + 64 * D + 8 + 128);
    return per_cu ? std::max(0, kLds / (per_cu + 1) + 1024 - kOwn) : 0;
}

template <int D, bool BF16>
void launch_d(const Attn4Args &a, const Attn4Plan &plan, hipStream_t st) {
    const dim3 grid((unsigned)plan.workgroups);
    if constexpr (D <= 128) {
        if (plan.prompt) {
            if (plan.prompt == 2)
                hipLaunchKernelGGL((attn4_kernel<D, BF16, 2, 4, 2>), grid, dim3(256), 0, st, a);
            else
                hipLaunchKernelGGL((attn4_kernel<D, BF16, 2, 4, 4>), grid, dim3(256), 0, st, a);
            return;
        }
        if (plan.wide) {
            hipLaunchKernelGGL((attn4_kernel<D, BF16, 1, 8, 8>), grid, dim3(512), 0, st, a);
            return;
        }
    }
    hipLaunchKernelGGL((attn4_kernel<D, BF16, 1, 4, 4>), grid, dim3(256),
                       spare_lds<D>(plan.per_cu), st, a);
    if (plan.splits > 1) {
        // few rows with many splits: whole workgroups of 1024 to a row
        const int64_t lines = a.N * a.heads;
        const int threads = plan.splits > 16 ? kJoinThreads : 256, slots = threads / (D / 4);
        int par = 1;
        while (par < slots && 2 * par < plan.splits) par *= 2;
        const int64_t per = slots / par;
        hipLaunchKernelGGL((attn4_join_kernel<D, BF16>),
                           dim3((unsigned)((lines + per - 1) / per)), dim3(threads), 0, st, a, par);
    }
}

}  // namespace

hipError_t launch_attn4(const Attn4Args &a, const Attn4Plan &p, int bf16, int dim, hipStream_t st) {
    if (dim == 64) { if (bf16) launch_d<64, true>(a, p, st); else launch_d<64, false>(a, p, st); }
    else if (dim == 128) { if (bf16) launch_d<128, true>(a, p, st); else launch_d<128, false>(a, p, st); }
    else { if (bf16) launch_d<256, true>(a, p, st); else launch_d<256, false>(a, p, st); }
    return hipGetLastError();
}

}  // namespace bitnet
