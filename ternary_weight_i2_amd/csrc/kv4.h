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

#include "common.h"

namespace bitnet {

constexpr int kPage = 64;    // tokens of a page
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

// The sequence of row r: the largest b with start[b] <= r (0 if there is none).
// Always in [0, n), whatever start holds.
__device__ __forceinline__ int64_t sequence_of(const int32_t *start, int64_t n, int64_t r) {
    int64_t lo = 0, hi = n - 1;
    while (lo < hi) {
        const int64_t m = (lo + hi + 1) >> 1;
        if (start[m] <= r) lo = m;
        else hi = m - 1;
    }
    return lo;
}

// Tokens of sequence b that the cache can hold: kv_len held to [0, 64 max_pages].
__device__ __forceinline__ int64_t held_tokens(const Kv4Args &c, int64_t b) {
    const int64_t t = c.kv_len[b], most = c.max_pages * kPage;
    return t < 0 ? 0 : t > most ? most : t;
}

// Row r of a call (a new token, or one to read): its place in the cache.
struct Kv4Place {
    int64_t rec;   // record index of kv head 0, or -1 if the row has no place
    int in_page;
};
__device__ __forceinline__ Kv4Place place_of(const Kv4Args &c, int64_t r) {
    Kv4Place p{-1, 0};
    const int64_t b = sequence_of(c.q_start, c.n_seqs, r);
    const int64_t first = c.q_start[b], end = c.q_start[b + 1];
    const int64_t held = held_tokens(c, b);
    const int64_t pos = held - (end - r);
    if (r < first || r >= end || pos < 0 || pos >= held) return p;
    const int64_t page = c.table[b * c.max_pages + pos / kPage];
    if (page < 0 || page >= c.n_pages) return p;
    p.rec = page * c.kv_heads;
    p.in_page = (int)(pos % kPage);
    return p;
}
// Whether row r belongs to one of the call's sequences at all.
__device__ __forceinline__ bool row_in_call(const Kv4Args &c, int64_t r) {
    return r >= c.q_start[0] && r < c.q_start[c.n_seqs];
}

}  // namespace bitnet
