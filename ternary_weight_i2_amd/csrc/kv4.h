// kv4.h -- the 4-bit key/value cache: its quantiser, the layout of a page
// record, and where a call's tokens are in it.
//
// A page holds 64 tokens; the record of one (page, kv head) is 72 * D bytes for
// D channels in G = D / 64 groups of 64:
//   0     key codes    [64 tokens][4 quads][D/32 steps][4 bytes]: the dword
//                      (quad, step) holds channels 32*step + 8*quad + 0..7,
//                      channel i in bits 4i..4i+3
//   32 D  value codes  [16 blocks of 4 tokens][16 lanes][G][4 tokens][2 bytes]:
//                      a halfword holds channels 64*g + 4*lane + 0..3
//   64 D  key pairs    [64 tokens][G] (step, middle), two fp16 numbers
//   68 D  value pairs  [16 blocks][G] (step x 4 tokens, middle x 4 tokens)
// so that the fragments of a 16x16x32 matrix instruction come straight out of
// wide loads: a key fragment is 8 channels of one token, D/32 of them side by
// side for a lane; a value fragment is 8 tokens of one channel, two tokens of
// four channels to a dword.
//
// A group's 64 values are quantised as
//   x is held to [-57344, 57344];  lo, hi: the smallest and largest
//   mid  = fp16(lo + (hi - lo) * fp32(8/15))
//   step = fp16(max((hi - mid) * fp32(1/7), (mid - lo) / 8))
//   code = clamp(round_half_even((x - mid) * fp32(1 / step) + 8), 0, 15), 8 if step is 0
//   value = mid + step * (code - 8)
// every operation one fp32 rounding.  step * (code - 8) is exact in fp32, and
// code - 8 costs one packed fp16 addition.
#pragma once

#include "layer.h"

namespace bitnet {

constexpr int kGroup = 64;   // channels that share a (step, middle) pair
constexpr float kKv4Max = 57344.0f;   // mid + 7 * step then stays below the largest fp16

template <int D>
struct Kv4Page {
    static constexpr int kGroups = D / kGroup;
    static constexpr int kSteps = D / 32;          // dwords of a token's quad
    static constexpr int kRow = D / 2;             // bytes of a token's codes
    static constexpr int kValues = 32 * D;
    static constexpr int kKeyPairs = 64 * D;
    static constexpr int kValuePairs = 68 * D;
    static constexpr int kBytes = 72 * D;
};

// Tiles of ROWS rows, a sequence's own from first_tile on: the sequence of tile x, the
// largest b for which that is at most x; its rows [begin,
// end) as q_start has them, and `held`, the tokens that the cache can hold of it,
// kv_len held to [0, 64 max_pages].  64 probes at a time, the same x in every lane;
// the last 64 bring the lengths with them, which saves a round trip.  The result is
// uniform and seq in [0, n_seqs), whatever the arrays hold.
struct SeqAt {
    int seq, begin, end, held;
};
template <int ROWS, int SLACK>
__device__ __forceinline__ SeqAt sequence_of(const Kv4Args &c, uint32_t G, uint32_t x) {
    const int lane = threadIdx.x & 63;
    auto at_most = [&](int b, int begin) { return first_tile<ROWS, SLACK>(begin, G, b) <= x; };
    int lo = 0, n = (int)c.n_seqs;   // the answer is in [lo, lo + n)
    while (n > 64) {
        const int step = (n + 63) >> 6, b = lo + lane * step;
        const bool ok = lane * step < n && at_most(b, c.q_start[b]);
        const int hits = __popcll(__ballot(ok));   // all probes up to the answer's
        const int k = hits > 0 ? hits - 1 : 0;
        lo += k * step;
        n = min(step, n - k * step);
    }
    const int b = lo + min(lane, n - 1);
    const int begin = c.q_start[b], end = c.q_start[b + 1], len = c.kv_len[b];
    const int hits = __popcll(__ballot(lane < n && at_most(b, begin)));
    const int k = __builtin_amdgcn_readfirstlane(hits > 0 ? hits - 1 : 0);
    const int64_t most = c.max_pages * kPage;   // up to 2^30
    return SeqAt{__builtin_amdgcn_readfirstlane(lo) + k, __builtin_amdgcn_readlane(begin, k),
                 __builtin_amdgcn_readlane(end, k),
                 min(max(__builtin_amdgcn_readlane(len, k), 0), (int)most)};
}

// Whether row r belongs to one of the call's sequences at all.
__device__ __forceinline__ bool row_in_call(const Kv4Args &c, int64_t r) {
    return r >= c.q_start[0] && r < c.q_start[c.n_seqs];
}

constexpr float kNoMax = -3.0e38f; // a running maximum before the first visible token

// The tile (ROWS rows of one sequence) that a workgroup works on, and the pages
// its rows see: the first `sink_pages`, then from `first` to the last.
struct Tile {
    int seq, token0, held;      // token0: the sequence's first query token
    uint32_t rows, row0;
    int pos0;                   // position of row 0's token
    int first, sink_pages, pages;
};

template <int ROWS>
__device__ __forceinline__ Tile find_tile(const Kv4Args &c, int64_t N, int window, int sinks,
                                          uint32_t x, uint32_t G) {
    Tile t;
    // a sequence has at least as many tiles to itself as its rows need
    const SeqAt s = sequence_of<ROWS, 1>(c, G, x);
    t.seq = s.seq;
    t.token0 = s.begin;
    const bool good = s.begin >= 0 && s.end > s.begin && s.end <= (int)N;
    t.rows = good ? (uint32_t)(s.end - s.begin) * G : 0;
    const int tile = (int)(x - first_tile<ROWS, 1>(s.begin, G, s.seq));
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
    t.first = window > 0 && pos_a >= window ? (pos_a - window + 1) / kPage : 0;
    t.sink_pages = min((sinks + kPage - 1) / kPage, t.first);
    t.pages = t.sink_pages + pos_b / kPage - t.first + 1;
    return t;
}

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
        x[e] = __builtin_amdgcn_fmed3f(x[e], -kKv4Max, kKv4Max);   // a NaN becomes -kKv4Max
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
    // Adding 1.5 * 2^23 rounds the held value to an integer, half to even, and
    // leaves it in the low bits above a constant; the constants of all eight are
    // taken off at once.
    constexpr uint32_t kMagic = 0x4b400000u;
    uint32_t codes = 0u - kMagic * 0x11111111u;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float t = (x[e] - mid) * inv;
        const float c = __builtin_amdgcn_fmed3f(t + 8.0f, 0.0f, 15.0f) + 12582912.0f;
        codes += __float_as_uint(c) << (4 * e);
    }
    *pair = (uint32_t)__builtin_bit_cast(uint16_t, step16) |
            (uint32_t)__builtin_bit_cast(uint16_t, mid16) << 16;
    return codes;
}

// The four positions [base, base + 4) of a workgroup, and their rows in the call.
struct Block4 {
    int page;           // its entry in the table (or -1): not looked at before a page is
    int in_page;        // of base: a multiple of 4
    int row;            // the call's row at base
    uint32_t rows;      // bit t: the call has a row at base + t
    int base, seq;      // its first position (negative: in front of the cache), its sequence
    __device__ bool cached(const Kv4Args &c) const { return page >= 0 && page < c.n_pages; }
};
__device__ __forceinline__ Block4 find_block(const Kv4Args &c, int64_t N) {
    Block4 k{-1, 0, 0, 0, 0, 0};
    const SeqAt s = sequence_of<4, 2>(c, 1, blockIdx.x);
    const int tile = (int)(blockIdx.x - first_tile<4, 2>(s.begin, 1, s.seq));
    if (tile < 0 || s.begin < 0 || s.end <= s.begin || s.end > N) return k;
    const int pos0 = s.held - (s.end - s.begin), base = (pos0 & ~3) + 4 * tile;
    k.row = s.begin + base - pos0;
    k.base = base;
    k.seq = s.seq;
    for (int t = 0; t < 4; ++t)
        if (base + t >= pos0 && base + t < s.held) k.rows |= 1u << t;
    if (base < 0 || !k.rows) return k;   // base is a multiple of 4: all four lie before 0
    k.page = c.table[s.seq * c.max_pages + base / kPage];
    k.in_page = base % kPage;
    return k;
}

// A lane's codes and pairs of eight channels (8 p on) of four tokens, t0 on, into their
// record: those tokens that `rows` has a bit for.
template <int D>
__device__ __forceinline__ void store_block4(uint8_t *rec, bool is_v, int t0, int p, uint32_t rows,
                                             const uint32_t (&codes)[4], const uint32_t (&pair)[4]) {
    using L = Kv4Page<D>;
    const int g = p >> 3;
    if (!is_v) {
        uint32_t *w = reinterpret_cast<uint32_t *>(rec) + t0 * (D / 8) + (p & 3) * L::kSteps + (p >> 2);
        uint32_t *m = reinterpret_cast<uint32_t *>(rec + L::kKeyPairs) + t0 * L::kGroups + g;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            if (!(rows >> t & 1)) continue;
            w[t * (D / 8)] = codes[t];
            if ((p & 7) == 0) m[t * L::kGroups] = pair[t];
        }
        return;
    }
    // halfwords [token] of this lane's two value lanes, and [step, mid][token]
    uint16_t *w = reinterpret_cast<uint16_t *>(rec + L::kValues) +
                  ((t0 >> 2) * 16 + 2 * (p & 7)) * L::kGroups * 4 + g * 4;
    uint16_t *m = reinterpret_cast<uint16_t *>(rec + L::kValuePairs) +
                  ((t0 >> 2) * L::kGroups + g) * 8;
    if (rows == 15) {
        auto low = [](uint32_t a, uint32_t b) { return (a & 0xffffu) | b << 16; };
        auto high = [](uint32_t a, uint32_t b) { return a >> 16 | (b & 0xffff0000u); };
        *reinterpret_cast<uint2 *>(w) = make_uint2(low(codes[0], codes[1]), low(codes[2], codes[3]));
        *reinterpret_cast<uint2 *>(w + 4 * L::kGroups) =
            make_uint2(high(codes[0], codes[1]), high(codes[2], codes[3]));
        if ((p & 7) == 0)
            *reinterpret_cast<uint4 *>(m) =
                make_uint4(low(pair[0], pair[1]), low(pair[2], pair[3]),
                           high(pair[0], pair[1]), high(pair[2], pair[3]));
        return;
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        if (!(rows >> t & 1)) continue;
        w[t] = (uint16_t)codes[t];
        w[4 * L::kGroups + t] = (uint16_t)(codes[t] >> 16);
        if ((p & 7) == 0) {
            m[t] = (uint16_t)pair[t];
            m[4 + t] = (uint16_t)(pair[t] >> 16);
        }
    }
}

}  // namespace bitnet
