// attn_plan.h -- which launch a call of the attention over the 4-bit cache takes
// (attn_kv4.hip: the kernels).  Host arithmetic on the call's sizes, without HIP.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace bitnet {

constexpr int kPage = 64;     // tokens of a page
constexpr int kUnits = 256;   // compute units
constexpr int kMaxSplits = 256;
constexpr int kPromptFrom = 2048, kPromptRows = 128;   // see attn4_plan
constexpr int64_t kAttn4Workgroups = 1 << 24;   // of 256 threads: a launch has fewer than 2^32

// Which kernel a call's sizes take (prompt: its tiles to a workgroup, or 0), how many
// workgroups share the pages of one row tile, how many may be on a compute unit at
// once (0: any), the tiles of a kv head and the workgroups of all.
struct Attn4Plan {
    int prompt, wide, splits, per_cu;
    int64_t tiles, workgroups;
};

// The pages of a split: an even share, of at least a page for every wave and, where
// it is short, the same number for each.
constexpr int chunk_of(int pages, int splits) {
    const int c = (int)((uint32_t)(pages + splits - 1) / (uint32_t)splits);
    return c >= 16 ? c : c <= 4 ? 4 : (c + 3) & ~3;
}

// Measured on the times of calls in a graph.
inline Attn4Plan attn4_plan(int64_t n_seqs, int64_t N, int64_t heads, int64_t kv_heads,
                            int64_t dim, int64_t max_kv, int64_t window, int64_t sinks,
                            bool bf16) {
    const int64_t rows = N * (heads / kv_heads), each = rows / 16 * kv_heads;
    int64_t pages = (max_kv + kPage - 1) / kPage;
    if (window > 0)   // what a tile's rows can see of it: the window before each, the sinks
        pages = std::min(pages, (window + 16) / kPage + 2 + (sinks + kPage - 1) / kPage);
    // Two fragments of rows to a wave, if there are enough workgroups without any
    // split and sequences have kPromptRows rows on average, so that tiles are full
    // (512 sequences of 8 rows at 1000 tokens: 89 us with one fragment, 119 with two;
    // of 128 rows 57 and 60 us either way round; 50 of 512 rows: 123 and 108).
    // Where one fragment would make kPromptFrom workgroups, two tiles to a workgroup
    // (those behind the last have no rows): three prompts of 2048, 16/8 heads of 128,
    // 92 -> 81 us when it was added; 700 rows of 32/8 heads from nothing 18 us with one
    // fragment, 21 with two.  Over long histories, where one fragment would make more
    // workgroups than run at once, all four waves on one tile: after 8000 tokens, 20/5
    // heads of 128, 640 rows 110 us with one fragment and 97 so, but 512 83 and 92; 2048
    // rows 292 us in pairs of tiles and 249 so, but a prompt of 4096 125 and 133.
    const bool lengthy = pages >= 32 && 32 * pages >= each;
    if (dim <= 128 && each >= (lengthy ? 3 * kUnits + 1 : kPromptFrom) &&
        rows >= kPromptRows * n_seqs) {
        const int at = lengthy ? 1 : 2;   // tiles to a workgroup
        const int64_t tiles = (rows / 32 + n_seqs + at - 1) / at * at;
        return Attn4Plan{at, 0, 1, 0, tiles, tiles / at * kv_heads};
    }
    const int64_t tiles = rows / 16 + n_seqs, groups = tiles * kv_heads;
    // A workgroup to a compute unit and a few pages to a wave: splitting costs more
    // than it saves (20/5 heads of 128, one token: fp32 9.4 us whole and 9.9 split at
    // 12 pages, 11.7 and 9.9 at 13; bf16 8.7 and 9.2 at 18, 10.2 and 9.1 at 21).
    const int64_t whole = bf16 ? 20 : 12;
    if (dim <= 128 && groups <= 256 && pages <= whole)
        return Attn4Plan{0, 1, 1, 0, tiles, groups};
    // Chunks of pages, so that a batch's workgroups are alike however its lengths
    // differ, for all the workgroups with rows (of sequences of one length) that run
    // at once, but none beyond: 32 sequences of 2000 tokens, 32/8 heads of 64 20.6 us
    // at four to a compute unit and 18.3 at three; 8 of 4000, heads of 128, fp32 18.0
    // at two, 21.1 at three.
    // Workgroups without rows, of sequences without any, cost time too, if little:
    // at most 64 of all for each page (256 sequences, of which 8 have a row at 500
    // tokens, 32/8 heads of 128: 14.9 -> 9.2 us; one at 4000: 53 -> 25; at 30000: 175
    // -> 61).
    const int64_t tall = (std::max<int64_t>(rows / n_seqs, 1) + 15) / 16;
    const int64_t busy = std::min(n_seqs, N) * tall * kv_heads;
    const int64_t at_once = kUnits * (dim == 64 ? 3 : dim == 256 && bf16 ? 1 : 2);
    const int64_t most = std::min<int64_t>({64 * pages / groups, kMaxSplits,
                                            (kAttn4Workgroups - 1) / groups});
    int64_t s = std::max<int64_t>(std::min(at_once / busy, most), 1);
    const int64_t chunk = chunk_of((int)pages, (int)s);
    s = std::max<int64_t>((pages + chunk - 1) / chunk, 1);
    // Up to two to a compute unit are kept at two: where three fit, the workgroups
    // without rows between them let some units take three and others one (64
    // sequences of 2000 tokens, 32/8 heads of 128, fp32 37.9 -> 32.2 us).  Whole
    // bf16 histories are bound by HBM and want the third (64 of 4095, 64/8 heads:
    // 43.3 us, held to two 49.9).
    const bool hold = dim == 128 && busy * s <= 2 * kUnits && (s > 1 || !bf16);
    return Attn4Plan{0, 0, (int)s, hold ? 2 : 0, tiles, groups * s};
}

}  // namespace bitnet
