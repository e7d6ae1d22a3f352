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

// Tiles of ROWS rows, a sequence's own from start[b] * G / ROWS + SLACK * b on: the
// sequence of tile x, the largest b for which that is at most x.  64 probes at a
// time, the same x in every lane; the result is uniform and always in [0, n),
// whatever start holds.
template <int ROWS, int SLACK>
__device__ __forceinline__ int sequence_of(const int32_t *start, int n, uint32_t G, uint32_t x) {
    const int lane = threadIdx.x & 63;
    int lo = 0;   // the answer is in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 63) >> 6, b = lo + lane * step;
        const bool ok = lane * step < n && (uint32_t)start[b] * G / ROWS + SLACK * b <= x;
        const int hits = __popcll(__ballot(ok));   // all probes up to the answer's
        const int k = hits > 0 ? hits - 1 : 0;
        lo += k * step;
        n = min(step, n - k * step);
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

// Tokens of sequence b that the cache can hold: kv_len held to [0, 64 max_pages].
__device__ __forceinline__ int64_t held_tokens(const Kv4Args &c, int64_t b) {
    const int64_t t = c.kv_len[b], most = c.max_pages * kPage;
    return t < 0 ? 0 : t > most ? most : t;
}

// Whether row r belongs to one of the call's sequences at all.
__device__ __forceinline__ bool row_in_call(const Kv4Args &c, int64_t r) {
    return r >= c.q_start[0] && r < c.q_start[c.n_seqs];
}

}  // namespace bitnet
