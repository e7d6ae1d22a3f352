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

// Tiles of ROWS rows, a sequence's own from start[b] * G / ROWS + SLACK * b on: the
// sequence of tile x, the largest b for which that is at most x; its rows [begin,
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
    auto at_most = [&](int b, int begin) { return (uint32_t)begin * G / ROWS + SLACK * b <= x; };
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

}  // namespace bitnet
