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

// The first of a sequence's own tiles of ROWS rows, G rows to a token: `begin` its first token in the
// call, SLACK the tiles that a sequence may have beyond its rows' share.
template <int ROWS, int SLACK>
constexpr uint32_t first_tile(int begin, uint32_t G, int seq) {
    return (uint32_t)begin * G / ROWS + (uint32_t)(SLACK * seq);
}

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

// kv4_weigh.hip: the tiles of 16 rows; the shares of the pages that a tile's rows see, and of a
// sequence's pages where its rows are few; whether rows are many (a workgroup to a page) and
// the parts that they are then in.
struct WeighPlan {
    int64_t tiles;
    int splits, chunks, many, parts;
    // the workspace: rows' maxima and sums, the queries as operands, the parts' sums
    int64_t kept_at, sums_at, bytes;
};
inline WeighPlan weigh_plan(int64_t n_seqs, int64_t N, int64_t heads, int64_t kv_heads,
                            int64_t dim, int64_t max_kv, int64_t window, int64_t sinks,
                            bool bf16) {
    // workgroups of a launch; more units take turns, so empty sequences make no more than these
    constexpr int64_t kMost = 1 << 22;
    const int64_t rows = N * (heads / kv_heads), pages = std::max<int64_t>((max_kv + kPage - 1) / kPage, 1);
    int64_t seen = pages;
    if (window > 0) seen = std::min(pages, (window + 16) / kPage + 2 + (sinks + kPage - 1) / kPage);
    WeighPlan p;
    p.tiles = rows / 16 + n_seqs;
    // Four workgroups to a compute unit and a page at least for every wave; at most 128 shares of
    // a tile, which each of its rows joins.  (Shares of a fixed number of pages, so that ragged
    // sequences have workgroups of one size, took longer: 64 sequences of 820 to 4096
    // tokens 70 us with 32 pages and 77 with 16, two even shares of each 62.)
    const int64_t tall = (std::max<int64_t>(rows / n_seqs, 1) + 15) / 16;
    const int64_t busy = std::min(n_seqs, N) * tall * kv_heads, few = std::min(n_seqs, N) * kv_heads;
    // (Of the call on average, which its sizes tell: kv4_weigh.hip has what that costs a mixed one.)
    p.many = rows >= 4 * 16 * n_seqs;
    p.splits = (int)std::max<int64_t>(
        std::min({4 * kUnits / busy, seen / 4, (int64_t)128, kMost / (p.tiles * kv_heads)}), 1);
    p.chunks = (int)std::max<int64_t>(
        std::min(p.many ? pages : std::min(pages / 4, 4 * kUnits / few), kMost / (n_seqs * kv_heads)), 1);
    // Where pages are few, their rows in parts of eight tiles or more, for 8 workgroups to a unit
    // (a prompt of 2048, 20/5 heads: 208 us whole, 47 so; 131 rows of 190 pages, of which a window
    // sees 66: 28 us whole, 37 in three).
    p.parts = p.many ? (int)std::max<int64_t>(
                           std::min(8 * kUnits / (n_seqs * p.chunks * kv_heads), tall / 8), 1)
                     : 1;
    const int64_t pieces = (bf16 ? 1 : 2) * dim / 32 + (dim == 256 ? 2 : 1);   // kept_pieces
    p.kept_at = (p.splits * N * heads * 8 + 15) / 16 * 16;
    p.sums_at = p.kept_at + (p.many ? p.tiles * kv_heads * pieces * 1024 : 0);
    p.bytes = p.sums_at + (p.parts > 1 ? n_seqs * p.chunks * kv_heads * p.parts * kPage * 4 : 0);
    return p;
}

// kv4_evict.hip: the workgroups that choose the tokens of a (sequence, kv head), and what they
// tell each other: bins of three passes, the search's state after each, counts of each slice.
constexpr int kBins = 2048;
constexpr int kEvictSlicesFrom = 320;   // pages: 32768 tokens 52 us by one, 34 by eight; 16384 35 by one
struct EvictPlan {
    int slices;
    int64_t search_at, slices_at, bytes;
};
inline EvictPlan evict_plan(int64_t n_seqs, int64_t kv_heads, int64_t max_pages) {
    const int64_t units = n_seqs * kv_heads;
    EvictPlan p{1, 0, 0, 0};
    // The table's width stands for the histories' lengths, which only the device has: 16 histories
    // of up to 2176 tokens, 8 heads, take 23.5 us with the move in a table of 34 entries and 50 in
    // one of 320 or more.
    // 131072 tokens of one head: 47 us by 16 workgroups, 49 by 32, 54 by 8; of eight: 71, 73, 78.
    if (max_pages >= kEvictSlicesFrom)
        p.slices = (int)std::max<int64_t>(std::min({max_pages / 64, 2 * kUnits / units, (int64_t)16}), 1);
    if (p.slices == 1) return p;
    p.search_at = 3 * units * p.slices * kBins * 4;
    p.slices_at = p.search_at + 3 * units * 8;
    p.bytes = p.slices_at + units * p.slices * 8;
    return p;
}
// The tokens [from, to) of a slice of a history of `held`.  `from` is a multiple of four also
// behind the end (where to <= from): threads load four weights at once from there on, whether
// they are the slice's or not, and four from a multiple of four on are in one page.
struct EvictSlice {
    int from, to;
};
constexpr EvictSlice evict_slice(int held, int slices, int slice) {
    const int share = ((held + slices - 1) / slices + 3) & ~3;   // held is at most 2^30
    const int end = (held + 3) & ~3, from = slice * share < end ? slice * share : end;
    return EvictSlice{from, from + share < held ? from + share : held};
}

}  // namespace bitnet
