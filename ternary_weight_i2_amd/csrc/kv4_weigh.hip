// kv4_weigh.hip -- the attention weight that each token of the 4-bit cache gets from a call's
// rows, added to what it had got before: what an eviction goes by.
//
//   out[t] = (t older than the rows ? decay * old[t] : 0) + sum_r p_rt,
//   p_rt = 2^(x_rt - m_r) / sum_s 2^(x_rs - m_r),   x_rt = log2(e) * scale * q_r . k_t
// summed over the rows of a sequence and the heads that share a kv head, whose queries are
// rows of one problem as in attn_kv4.hip.
//
// Two launches or three.  The first gives each row's maximum m and sum, a workgroup to 16 rows and
// a share of the pages that they see, its waves taking turns at the pages.  The second sums
// by token.  Few rows: `chunks` workgroups have a sequence's pages, a wave every (4 chunks)-th
// of the whole history, and go through the sequence's tiles of 16 rows one after another.  Many
// rows, 64 to a sequence or more: a workgroup to a page, its waves taking turns at the tiles
// that see it; where pages are few, several workgroups to a page, each with a part of these
// tiles, and a third launch adds the parts.  So no number is added to by two waves at once and
// the order of the sums is fixed.  The keys are read by both launches.
// Between them lie 8 bytes a row and share of the pages; of many rows also the queries as
// operands (a tile of 16 rows and kv head: 5 KB with bf16 heads of 128, 9 KB with fp32), most of
// a prompt's workspace; and 256 bytes a page, kv head and part.
//
// The form is the whole call's, by the rows of a sequence on average: one long chunk among many
// single tokens has few workgroups, which take its tiles one after another (255 tokens over 600
// to 2000 and one chunk of 512 over 4096, 32/8 heads of 128, bf16: 2460 us; the tokens by
// themselves 89, the chunk 109).  Two calls are the way there.
//
// q . k_t = sum_g step_tg (q_g . (code_tg - 8)) + mid_tg sum(q_g), the products of codes on
// the fp16 matrix instruction (q scaled by a power of two a row, in two fp16 terms of 22
// bits for fp32 rows, exactly for bf16 ones), all else in fp32.
//
// What bounds it: 64 tokens over up to 4096, 64/8 heads of 128, bf16, take 26 + 30 us for 88 MB of
// keys each time: workgroups of 820 to 4096 tokens that start together, each with a chain of
// five dependent loads, and about 280 vector operations a page (two pages asked for ahead made it
// 62 us in place of 60).  131 fp32 rows of 20/5 heads that see 66 pages: 22 + 28 us, vector operations and, in
// the second launch, 660 workgroups where 512 fit.  A prompt of 2048, 20/5 heads, bf16: 45 + 47 +
// 4 us, vector operations.
#include <algorithm>
#include <type_traits>

#include "codes4.h"
#include "kv4.h"

namespace bitnet {

namespace {

constexpr int kWeighThreads = 256;
constexpr int kWeighWaves = kWeighThreads / 64;

// Waves to a SIMD: what the registers of a head hold beside the page asked for ahead (64 bf16
// tokens, heads of 128: 61 us in all with three, 64.5 with four, which spilled).
constexpr int least_waves(int dim) { return dim == 256 ? 2 : dim == 128 ? 3 : 4; }

// A row's query: 8 channels of every 32 in this lane (quad), times 2^k; the sums of its
// groups at the same scale; and what makes a product of them a power of two's exponent.
template <int D, bool BF16>
struct Query {
    static constexpr int NT = BF16 ? 1 : 2, NS = D / 32, NG = D / 64;
    h8 f[NT][NS];
    float sum[NG], scale;
};
template <int D, bool BF16>
struct RawQuery {   // as it is loaded
    static constexpr int NW = BF16 ? 1 : 2;
    uint4 v[D / 32][NW];
};
template <int D, bool BF16>
__device__ __forceinline__ void load_query(RawQuery<D, BF16> &r, const void *p, int64_t at) {
    constexpr int NW = RawQuery<D, BF16>::NW;
#pragma unroll
    for (int j = 0; j < D / 32; ++j)
#pragma unroll
        for (int k = 0; k < NW; ++k) r.v[j][k] = reinterpret_cast<const uint4 *>(p)[(at + 32 * j) * NW / 8 + k];
}
template <int D, bool BF16>
__device__ __forceinline__ void make_query(Query<D, BF16> &q, const RawQuery<D, BF16> &r, float scale_log2) {
    using Q = Query<D, BF16>;
    float v[Q::NS][8], top = 0.0f;
#pragma unroll
    for (int j = 0; j < Q::NS; ++j) load8<BF16>(r.v[j], 0, v[j]);
#pragma unroll
    for (int j = 0; j < Q::NS; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[j][e]));
    top = quad_max(top);
    const int k = top > 0.0f ? min(15 - __builtin_amdgcn_frexp_expf(top), 126) : 0;
    const float up = ldexpf(1.0f, k);
    q.scale = ldexpf(scale_log2, -k);
#pragma unroll
    for (int g = 0; g < Q::NG; ++g) {
        float sum = 0.0f;
#pragma unroll
        for (int j = 2 * g; j < 2 * g + 2; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float z = v[j][(e >> 1) + 4 * (e & 1)] * up;
                const _Float16 hi = (_Float16)z;
                q.f[0][j][e] = hi;
                if constexpr (!BF16) q.f[1][j][e] = (_Float16)(z - (float)hi);
                sum += z;
            }
        q.sum[g] = quad_sum(sum);
    }
}

// Queries as the first launch leaves them for a second one of many rows: [tile][16 bytes
// of `Query`][lane] and, behind the operands, the scale and the sums.
template <int D, bool BF16>
constexpr int kept_pieces = Query<D, BF16>::NT * Query<D, BF16>::NS + (D == 256 ? 2 : 1);
template <int D, bool BF16>
__device__ __forceinline__ void keep_query(uint4 *p, const Query<D, BF16> &q, int lane) {
    using Q = Query<D, BF16>;
#pragma unroll
    for (int t = 0; t < Q::NT; ++t)
#pragma unroll
        for (int j = 0; j < Q::NS; ++j) p[(t * Q::NS + j) * 64 + lane] = __builtin_bit_cast(uint4, q.f[t][j]);
    uint32_t w[8] = {__float_as_uint(q.scale)};
#pragma unroll
    for (int g = 0; g < Q::NG; ++g) w[1 + g] = __float_as_uint(q.sum[g]);
    p[Q::NT * Q::NS * 64 + lane] = make_uint4(w[0], w[1], w[2], w[3]);
    if constexpr (D == 256) p[(Q::NT * Q::NS + 1) * 64 + lane] = make_uint4(w[4], w[5], w[6], w[7]);
}
template <int D, bool BF16>
__device__ __forceinline__ void kept_query(Query<D, BF16> &q, const uint4 *p, int lane) {
    using Q = Query<D, BF16>;
#pragma unroll
    for (int t = 0; t < Q::NT; ++t)
#pragma unroll
        for (int j = 0; j < Q::NS; ++j) q.f[t][j] = __builtin_bit_cast(h8, p[(t * Q::NS + j) * 64 + lane]);
    const uint4 a = p[Q::NT * Q::NS * 64 + lane];
    q.scale = __uint_as_float(a.x);
    q.sum[0] = __uint_as_float(a.y);
    if constexpr (Q::NG > 1) q.sum[1] = __uint_as_float(a.z);
    if constexpr (Q::NG > 2) {
        q.sum[2] = __uint_as_float(a.w);
        q.sum[3] = __uint_as_float(p[(Q::NT * Q::NS + 1) * 64 + lane].x);
    }
}

// A page's keys as they are loaded: this lane's codes of tokens 16 i + n, 8 channels of
// every 32, and the pairs of token `lane`, which the wave shares through LDS.
template <int D>
struct Keys {
    static constexpr int NS = D / 32, NG = D / 64;
    uint32_t code[4][NS], pair[NG];
};
template <int D>
__device__ __forceinline__ void load_keys(Keys<D> &k, const uint8_t *rec, int lane) {
    using L = Kv4Page<D>;
    const int n = lane & 15, quad = lane >> 4;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        load_words(rec + (16 * i + n) * L::kRow + quad * (D / 8), k.code[i]);
    const uint32_t *p = reinterpret_cast<const uint32_t *>(rec + L::kKeyPairs) + lane * L::kGroups;
#pragma unroll
    for (int g = 0; g < L::kGroups; ++g) k.pair[g] = p[g];
}
// The page's pairs into the wave's part of the LDS.
template <int D>
__device__ __forceinline__ void share_pairs(const Keys<D> &k, uint32_t *pairs, int lane) {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int g = 0; g < Keys<D>::NG; ++g) pairs[lane * Keys<D>::NG + g] = k.pair[g];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}
// A tile of eight rows at most has each of them in two of its 16 columns (REP 2), and each of
// their lanes works on its own half of a page's tokens behind the products: lane n has row
// n % (16 / REP) and the tokens 16 i + 4 quad + e of 4 / REP i, from first_of<REP>(n) on.  64
// bf16 tokens, 64/8 heads of 128: 60.2 us in all without, 55.6 so.  With fp32 rows the registers
// do not do (one token over 131072, 20/5 heads: 43 and 48 us, spills), nor with heads of 256; four
// rows four times took 48.9 there, and 16.1 for 15.5 us with heads of 64.
template <int D, bool BF16>
constexpr bool kTwice = BF16 && D <= 128;
template <int D, bool BF16>
__device__ __forceinline__ int rep_of(uint32_t left) { return kTwice<D, BF16> && left <= 8 ? 2 : 1; }
template <int REP>
__device__ __forceinline__ int first_of(int n) { return n / (16 / REP) * (4 / REP); }
template <int REP>
using Rep = std::integral_constant<int, REP>;

// x / q.scale of token 16 i + 4 quad + e and this lane's row, in s[i - first_of][e].
template <int REP, int D, bool BF16>
__device__ __forceinline__ void scores(const Keys<D> &k, const uint32_t *pairs, const Query<D, BF16> &q,
                                       uint32_t one, int n, int quad, float (&s)[4 / REP][4]) {
    using Q = Query<D, BF16>;
#pragma unroll
    for (int i = 0; i < 4 / REP; ++i) {
        f4 acc[Q::NG];
#pragma unroll
        for (int g = 0; g < Q::NG; ++g)
#pragma unroll
            for (int part = 0; part < REP; ++part) {
                f4 of_part = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int j = 2 * g; j < 2 * g + 2; ++j) {
                    h2 c[4];
                    codes8<false>(k.code[part * (4 / REP) + i][j], one, c);
                    const h8 kc = join(c[0], c[1], c[2], c[3]);
#pragma unroll
                    for (int t = 0; t < Q::NT; ++t) of_part = mfma(kc, q.f[t][j], of_part);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[g][e] = part == 0 || n / (16 / REP) == part ? of_part[e] : acc[g][e];
            }
        const int token = 16 * (first_of<REP>(n) + i) + 4 * quad;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float x = 0.0f;
#pragma unroll
            for (int g = 0; g < Q::NG; ++g) {
                const h2 p = as_h2(pairs[(token + e) * Q::NG + g]);   // (step, middle)
                x = fmaf((float)p[0], acc[g][e], fmaf((float)p[1], q.sum[g], x));
            }
            s[i][e] = x;
        }
    }
}

// Hides what a row at `pos`, whose window begins at `low`, does not see of page t0.
template <int REP>
__device__ __forceinline__ void hide(float (&s)[4 / REP][4], int t0, int n, int quad, int pos, int low, int sinks) {
#pragma unroll
    for (int i = 0; i < 4 / REP; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int j = t0 + 16 * (first_of<REP>(n) + i) + 4 * quad + e;
            const bool hidden = (j > pos) | ((j < low) & (j >= sinks));
            s[i][e] = hidden ? -INFINITY : s[i][e];
        }
}

// The pages of a tile's list (find_tile) that a wave takes, every kWeighWaves-th from `from`
// on: those that are there, 64 table entries at a time, one a lane.
struct Walk {
    const int32_t *table;
    int64_t n_pages;
    int first, sink_pages, from, end, mine, id;
    uint64_t there;
    __device__ int page_at(int i) const { return i < sink_pages ? i : first + i - sink_pages; }
    __device__ void entries() {
        const int i = from + kWeighWaves * (int)(threadIdx.x & 63);
        mine = i < end ? table[page_at(i)] : -1;
        there = __ballot(mine >= 0 && mine < n_pages);
    }
    // The next page's first token, or -1; `id` stays one that can be loaded.
    __device__ int next() {
        while (there == 0) {
            if (from >= end - 64 * kWeighWaves) return -1;
            from += 64 * kWeighWaves;
            entries();
        }
        const int bit = __builtin_ctzll(there);
        there &= there - 1;
        id = __builtin_amdgcn_readlane(mine, bit);
        return page_at(from + kWeighWaves * bit) * kPage;
    }
};
__device__ __forceinline__ Walk walk_of(const Kv4Args &c, const Tile &t, int begin, int end, int wave) {
    Walk w{c.table + (int64_t)t.seq * c.max_pages, c.n_pages, t.first, t.sink_pages, begin + wave, end, -1, 0, 0};
    w.entries();
    return w;
}

// What of a page t0 all 16 rows see, or none needs to be hidden from: the first row's
// position and the last row's window.
struct Seen {
    int pos_first, low_last, sinks;
    __device__ bool all(int t0) const {
        return t0 + kPage - 1 <= pos_first && (t0 >= low_last || t0 + kPage <= sinks);
    }
};
__device__ __forceinline__ Seen seen_of(const WeighArgs &a, const Tile &t, uint32_t G) {
    const uint32_t last = min(t.row0 + 15, t.rows - 1);
    return Seen{t.pos0 + (int)(t.row0 / G), a.window > 0 ? t.pos0 + (int)(last / G) - a.window + 1 : 0, a.sinks};
}

// The pages of one of `shares` even shares, at least one for every wave.
__device__ __forceinline__ int share_of(int pages, int shares) {
    return max((int)((uint32_t)(pages + shares - 1) / (uint32_t)shares), kWeighWaves);
}

template <int D, bool BF16>
__global__ __launch_bounds__(kWeighThreads, least_waves(D)) void weigh_stats_kernel(const WeighArgs a, int64_t units) {
    using L = Kv4Page<D>;
    __shared__ float m_all[kWeighWaves][16], l_all[kWeighWaves][16];
    __shared__ __align__(16) uint32_t pairs_all[kWeighWaves][D];
    const int lane = threadIdx.x & 63, n = lane & 15, quad = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t G = (uint32_t)a.heads / (uint32_t)a.c.kv_heads;
    const uint32_t one = ones_1024();
    for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
        // heads first, then the shares of a tile, then tiles
        const int64_t u = unit / a.c.kv_heads;
        const int kv_head = (int)(unit - u * a.c.kv_heads), split = (int)(u % a.splits);
        const Tile t = find_tile<16>(a.c, a.N, a.window, a.sinks, (uint32_t)(u / a.splits), G);
        if (t.rows == 0) continue;   // the whole workgroup
        const int rep = rep_of<D, BF16>(t.rows - t.row0);
        const uint32_t row = min(t.row0 + (n & (16 / rep - 1)), t.rows - 1), tok = row / G;
        const int head = kv_head * (int)G + (int)(row - tok * G);
        const int64_t line = (int64_t)(t.token0 + (int)tok) * a.heads + head;
        const int share = share_of(t.pages, a.splits), begin = min(split * share, t.pages), end = min(begin + share, t.pages);
        float m = kNoMax, l = 0.0f;
        if (begin < end) {
            Walk w = walk_of(a.c, t, begin, end, wave);
            const uint8_t *cache = a.c.cache + (int64_t)kv_head * L::kBytes;
            const int64_t page_bytes = (int64_t)a.c.kv_heads * L::kBytes;
            int t0 = w.next();
            Keys<D> k;
            load_keys(k, cache + w.id * page_bytes, lane);
            RawQuery<D, BF16> raw;
            load_query(raw, a.q, (t.token0 + (int64_t)tok) * a.q_stride + head * D + 8 * quad);
            Query<D, BF16> q;
            make_query(q, raw, a.scale_log2);
            if (a.kept && split == 0 && wave == 0)
                keep_query(a.kept + ((u / a.splits) * a.c.kv_heads + kv_head) * (kept_pieces<D, BF16> * 64), q, lane);
            const int pos = t.pos0 + (int)tok, low = a.window > 0 ? pos - a.window + 1 : 0;
            const Seen seen = seen_of(a, t, G);
            auto walk = [&](auto reps) {
                constexpr int REP = decltype(reps)::value;
                while (t0 >= 0) {
                    share_pairs(k, pairs_all[wave], lane);
                    const int t1 = w.next();   // a page is always loaded, at the end the last one again
                    Keys<D> ahead;
                    load_keys(ahead, cache + w.id * page_bytes, lane);
                    float s[4 / REP][4];
                    scores<REP>(k, pairs_all[wave], q, one, n, quad, s);
                    if (!seen.all(t0)) {
                        asm volatile("");   // a branch: most pages are seen by all rows
                        hide<REP>(s, t0, n, quad, pos, low, a.sinks);
                    }
                    float top = -INFINITY;
#pragma unroll
                    for (int i = 0; i < 4 / REP; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) top = fmaxf(top, s[i][e]);
                    const float m_new = fmaxf(m, top * q.scale);
                    l *= __builtin_amdgcn_exp2f(m - m_new);
                    m = m_new;
#pragma unroll
                    for (int i = 0; i < 4 / REP; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) l += __builtin_amdgcn_exp2f(fmaf(s[i][e], q.scale, -m));
                    t0 = t1;
                    k = ahead;
                }
            };
            if (kTwice<D, BF16> && rep == 2) walk(Rep<kTwice<D, BF16> ? 2 : 1>{});
            else walk(Rep<1>{});
        }
        // a row's four lanes, then the waves
        const float top = quad_max(m);
        l = quad_sum(l * __builtin_amdgcn_exp2f(m - top));
        __syncthreads();   // the last unit's have been read
        if (quad == 0) {
            m_all[wave][n] = top;
            l_all[wave][n] = l;
        }
        __syncthreads();
        if ((int)threadIdx.x < 16 / rep && t.row0 + n < t.rows) {
            float best = m_all[0][n], sum = 0.0f;
            for (int c = n; c < 16; c += 16 / rep)   // the row's columns
#pragma unroll
                for (int w = 0; w < kWeighWaves; ++w) best = fmaxf(best, m_all[w][c]);
            for (int c = n; c < 16; c += 16 / rep)
#pragma unroll
                for (int w = 0; w < kWeighWaves; ++w)
                    sum = fmaf(l_all[w][c], __builtin_amdgcn_exp2f(m_all[w][c] - best), sum);
            a.part[split * a.N * a.heads + line] = make_float2(best, sum);
        }
    }
}

// A row's maximum and one over its sum; 0 for a row that sees nothing, is no number or none
// of the tile's.
struct Row {
    float max, inv;
};
__device__ __forceinline__ Row row_of(const WeighArgs &a, int64_t line, bool real, int quad) {
    // the four lanes of a row take turns at its shares, four loads at a time
    const int64_t stride = a.N * a.heads;
    float m = kNoMax, l = 0.0f;
    for (int s0 = quad; s0 < a.splits; s0 += 16) {
        float2 o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = a.part[min(s0 + 4 * i, a.splits - 1) * stride + line];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (s0 + 4 * i >= a.splits) continue;
            const float best = fmaxf(m, o[i].x);
            l = l * __builtin_amdgcn_exp2f(m - best) + o[i].y * __builtin_amdgcn_exp2f(o[i].x - best);
            m = best;
        }
    }
    const float best = quad_max(m);
    l = quad_sum(l * __builtin_amdgcn_exp2f(m - best));
    const bool good = real && l > 0.0f && l < INFINITY;
    return Row{good ? best : 0.0f, good ? 1.0f / l : 0.0f};
}
template <int N>
__device__ __forceinline__ void add_weights(float (&x)[N][4], float scale, const Row &r, float (&w)[N][4]) {
    if (__any(r.inv == 0.0f))   // their scores may be no numbers
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[i][e] = r.inv > 0.0f ? x[i][e] : 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            w[i][e] = fmaf(__builtin_amdgcn_exp2f(fmaf(x[i][e], scale, -r.max)), r.inv, w[i][e]);
}
// Over the 16 rows; lane n of a quad keeps token 16 (n / 4) + 4 quad + n % 4: lanes hand each
// other the half of the values that the other keeps, but for what they have not (REP).
template <int CTRL, int HALF, int N>
__device__ __forceinline__ void fold(float (&v)[N], bool upper) {
#pragma unroll
    for (int k = 0; k < HALF; ++k) {
        const float keep = upper ? v[k + HALF] : v[k], give = upper ? v[k] : v[k + HALF];
        v[k] = keep + dpp_f32<CTRL>(give);
    }
}
template <int N>
__device__ __forceinline__ float sum_rows(const float (&w)[N][4], int n) {
    float v[4 * N];
#pragma unroll
    for (int k = 0; k < 4 * N; ++k) v[k] = w[k >> 2][k & 3];
    if constexpr (N == 4) fold<kDppMirror, 8>(v, n & 8);
    if constexpr (N >= 2) fold<kDppHalfMirror, 4>(v, n & 4);
    fold<kDppXor2, 2>(v, n & 2);
    fold<kDppXor1, 1>(v, n & 1);
    return v[0];
}
__device__ __forceinline__ int place_of(int lane) {
    return 16 * ((lane & 15) >> 2) + 4 * (lane >> 4) + (lane & 3);
}

// Few rows: `chunks` workgroups have a sequence's pages, their waves taking turns, and a tile's
// queries stay in registers.  The pages that the first tile does not see get their
// old weights; what another tile adds, it adds to what its own lanes have written.
template <int D, bool BF16>
__global__ __launch_bounds__(kWeighThreads, least_waves(D)) void weigh_few_kernel(const WeighArgs a, int chunks, int64_t units) {
    using L = Kv4Page<D>;
    __shared__ __align__(16) uint32_t pairs_all[kWeighWaves][D];
    const int lane = threadIdx.x & 63, n = lane & 15, quad = lane >> 4, place = place_of(lane);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t G = (uint32_t)a.heads / (uint32_t)a.c.kv_heads;
    const uint32_t one = ones_1024();
    for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const int64_t u = unit / a.c.kv_heads;
        const int kv_head = (int)(unit - u * a.c.kv_heads), seq = (int)(u / chunks), part = (int)(u - (int64_t)seq * chunks);
        const int begin = a.c.q_start[seq], end = a.c.q_start[seq + 1];
        const int held = min(max(a.c.kv_len[seq], 0), (int)(a.c.max_pages * kPage));
        if (begin < 0 || end <= begin || end > a.N) continue;   // the whole workgroup
        const int pages = (held + kPage - 1) / kPage;
        const int pos0 = held - (end - begin);
        const uint32_t rows = (uint32_t)(end - begin) * G;
        const int32_t *table = a.c.table + (int64_t)seq * a.c.max_pages;
        const uint8_t *cache = a.c.cache + (int64_t)kv_head * L::kBytes;
        const int64_t page_bytes = (int64_t)a.c.kv_heads * L::kBytes;
        auto weight_at = [&](int id) { return ((int64_t)id * a.c.kv_heads + kv_head) * kPage + place; };
        // A wave has every stride-th page, whichever tile sees it, so what it adds to has been
        // written by itself, and a window's pages are spread over the workgroups.
        const int stride = kWeighWaves * chunks;
        for (uint32_t r = 0; r * 16 < rows; ++r) {
            const uint32_t row0 = r * 16, last = min(row0 + 15, rows - 1);
            const int rep = rep_of<D, BF16>(rows - row0);
            const uint32_t mine = row0 + (n & (16 / rep - 1)), row = min(mine, last), tok = row / G;
            const int pos_a = pos0 + (int)(row0 / G), pos_b = pos0 + (int)(last / G);
            // the pages that its rows see: [0, sink_end) and [win, see_end)
            const int see_end = pos_b < 0 ? 0 : min(pos_b / kPage + 1, pages);
            const int win = a.window > 0 && pos_a >= a.window ? (pos_a - a.window + 1) / kPage : 0;
            const int sink_end = min((a.sinks + kPage - 1) / kPage, win);
            auto sees = [&](int p) { return p < sink_end || (p >= win && p < see_end); };
            const int head = kv_head * (int)G + (int)(row - tok * G);
            const int pos = pos0 + (int)tok, low = a.window > 0 ? pos - a.window + 1 : 0;
            Row rs{0.0f, 0.0f};
            Query<D, BF16> q;
            bool have = false;
            for (int from = part * kWeighWaves + wave; from < pages; from += 64 * stride) {
                const int i = from + stride * lane;
                const int ids = i < pages ? table[i] : -1;
                const uint64_t there = __ballot(ids >= 0 && ids < a.c.n_pages);
                uint64_t seen = __ballot(i < pages && sees(i)) & there;
                uint64_t rest = r == 0 ? there & ~seen : 0;
                if (seen) {
                    auto page = [&](uint64_t &bits, int &id) {   // the next one of them, or the last again
                        if (!bits) return -1;
                        const int bit = __builtin_ctzll(bits);
                        bits &= bits - 1;
                        id = __builtin_amdgcn_readlane(ids, bit);
                        return (from + stride * bit) * kPage;
                    };
                    int id = 0, t0 = page(seen, id);
                    Keys<D> k;
                    load_keys(k, cache + id * page_bytes, lane);
                    if (!have) {
                        have = true;
                        RawQuery<D, BF16> raw;
                        load_query(raw, a.q, (begin + (int64_t)tok) * a.q_stride + head * D + 8 * quad);
                        rs = row_of(a, (int64_t)(begin + (int)tok) * a.heads + head, mine < rows, quad);
                        make_query(q, raw, a.scale_log2);
                    }
                    const Seen all{pos_a, a.window > 0 ? pos_b - a.window + 1 : 0, a.sinks};
                    auto walk = [&](auto reps) {
                        constexpr int REP = decltype(reps)::value;
                        while (t0 >= 0) {
                            const int64_t at = weight_at(id);
                            const bool write = t0 + place < held;
                            float was = 0.0f, factor = 1.0f;
                            if (write) {
                                if (r > 0) was = a.out[at];
                                else if (t0 + place < pos0 && a.decay != 0.0f) was = a.old[at], factor = a.decay;
                            }
                            share_pairs(k, pairs_all[wave], lane);
                            const int t1 = page(seen, id);
                            Keys<D> ahead;
                            load_keys(ahead, cache + id * page_bytes, lane);
                            float x[4 / REP][4], w[4 / REP][4] = {};
                            scores<REP>(k, pairs_all[wave], q, one, n, quad, x);
                            if (!all.all(t0)) {
                                asm volatile("");
                                hide<REP>(x, t0, n, quad, pos, low, a.sinks);
                            }
                            add_weights(x, q.scale, rs, w);
                            const float sum = sum_rows(w, n);
                            if (write) a.out[at] = fmaf(factor, was, sum);
                            t0 = t1;
                            k = ahead;
                        }
                    };
                    if (kTwice<D, BF16> && rep == 2) walk(Rep<kTwice<D, BF16> ? 2 : 1>{});
                    else walk(Rep<1>{});
                }
                while (rest) {   // pages that no row of the first tile sees, four at a time
                    int64_t at[4];
                    float was[4];
                    bool write[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int bit = rest ? __builtin_ctzll(rest) : 0, t0 = (from + stride * bit) * kPage;
                        at[e] = weight_at(__builtin_amdgcn_readlane(ids, bit));
                        // (weights that stay are not written)
                        write[e] = rest && t0 + place < held && !(a.out == a.old && a.decay == 1.0f && t0 + kPage <= pos0);
                        was[e] = write[e] && t0 + place < pos0 && a.decay != 0.0f ? a.old[at[e]] : 0.0f;
                        rest &= rest - 1;
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (write[e]) a.out[at[e]] = a.decay * was[e];
                }
            }
        }
    }
}

// Many rows: a workgroup to a page and, where pages are few, to one of `parts` parts of the
// rows that see it, whose sums are then left in a.sums; its waves take turns at the tiles.
template <int D, bool BF16>
__global__ __launch_bounds__(kWeighThreads, 2) void weigh_many_kernel(const WeighArgs a, int chunks, int parts,
                                                                      int64_t units) {
    using L = Kv4Page<D>;
    __shared__ float w_all[kWeighWaves][64];
    __shared__ __align__(16) uint32_t pairs_all[kWeighWaves][D];
    const int lane = threadIdx.x & 63, n = lane & 15, quad = lane >> 4, place = place_of(lane);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t G = (uint32_t)a.heads / (uint32_t)a.c.kv_heads;
    const uint32_t one = ones_1024();
    for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const int64_t v = unit / parts, u = v / a.c.kv_heads;
        const int part = (int)(unit - v * parts), kv_head = (int)(v - u * a.c.kv_heads);
        const int seq = (int)(u / chunks), chunk = (int)(u - (int64_t)seq * chunks);
        const int begin = a.c.q_start[seq], end = a.c.q_start[seq + 1];
        const int held = min(max(a.c.kv_len[seq], 0), (int)(a.c.max_pages * kPage));
        if (begin < 0 || end <= begin || end > a.N) continue;   // the whole workgroup
        const int pos0 = held - (end - begin);
        const uint32_t rows = (uint32_t)(end - begin) * G;
        const uint32_t tile0 = first_tile<16, 1>(begin, G, seq);   // as the first launch has them (find_tile)
        for (int t0 = chunk * kPage; t0 < held; t0 += chunks * kPage) {
            const int id = a.c.table[seq * a.c.max_pages + t0 / kPage];
            if (id < 0 || id >= a.c.n_pages) continue;   // the whole workgroup
            // the rows that see the page: from position t0 on, and not beyond the window
            uint32_t r0 = t0 > pos0 ? (uint32_t)(t0 - pos0) * G / 16 : 0, r1 = (rows + 15) / 16;
            if (a.window > 0 && t0 >= a.sinks) {
                const int64_t last = (int64_t)t0 + kPage - 1 + a.window - 1 - pos0;   // the last token that does
                r1 = last < 0 ? 0 : (uint32_t)min((int64_t)r1, ((last + 1) * G + 15) / 16);
            }
            // (pages beyond the expected ones have no place for parts)
            const bool whole = parts == 1 || t0 >= chunks * kPage;
            if (whole && part > 0) continue;
            if (!whole && r0 < r1) {
                const uint32_t share = (r1 - r0 + parts - 1) / parts;
                r0 = min(r0 + part * share, r1);
                r1 = min(r0 + share, r1);
            }
            float w[4][4] = {};
            if (r0 < r1) {
                Keys<D> k;
                load_keys(k, a.c.cache + ((int64_t)id * a.c.kv_heads + kv_head) * L::kBytes, lane);
                // a tile's queries are on their way while those before are worked on
                Query<D, BF16> next;
                auto ask = [&](uint32_t r) {
                    kept_query(next, a.kept + ((int64_t)(tile0 + r) * a.c.kv_heads + kv_head) * (kept_pieces<D, BF16> * 64), lane);
                };
                ask(min(r0 + wave, r1 - 1));
                share_pairs(k, pairs_all[wave], lane);
                for (uint32_t r = r0 + wave; r < r1; r += kWeighWaves) {
                    uint32_t o = one;
                    if constexpr (D == 256) asm volatile("" : "+v"(o));   // unpacked again: too many to be kept
                    const uint32_t mine = r * 16 + n, last = min(r * 16 + 15, rows - 1), row = min(mine, last), tok = row / G;
                    const Row rs = row_of(a, (begin + (int64_t)tok) * a.heads + kv_head * (int)G + (int)(row - tok * G),
                                          mine < rows, quad);
                    const Query<D, BF16> q = next;
                    ask(min(r + kWeighWaves, r1 - 1));
                    const int pos = pos0 + (int)tok, low = a.window > 0 ? pos - a.window + 1 : 0;
                    float x[4][4];
                    scores<1>(k, pairs_all[wave], q, o, n, quad, x);
                    const Seen all{pos0 + (int)(r * 16 / G), a.window > 0 ? pos0 + (int)(last / G) - a.window + 1 : 0, a.sinks};
                    if (!all.all(t0)) {
                        asm volatile("");
                        hide<1>(x, t0, n, quad, pos, low, a.sinks);
                    }
                    add_weights(x, q.scale, rs, w);
                }
            }
            __syncthreads();   // the last page's have been read
            w_all[wave][place] = sum_rows(w, n);
            __syncthreads();
            if (wave == 0 && t0 + place < held) {
                float sum = w_all[0][place];
                for (int i = 1; i < kWeighWaves; ++i) sum += w_all[i][place];
                const int64_t at = ((int64_t)id * a.c.kv_heads + kv_head) * kPage + place;
                if (!whole) {
                    a.sums[unit * kPage + place] = sum;
                } else {
                    if (t0 + place < pos0 && a.decay != 0.0f) sum = fmaf(a.decay, a.old[at], sum);
                    a.out[at] = sum;
                }
            }
        }
    }
}

// The parts' sums, in their order, and the old weights: a wave to a page.
__global__ __launch_bounds__(kWeighThreads) void weigh_join_kernel(const WeighArgs a, int chunks, int parts, int64_t units) {
    const int place = threadIdx.x & 63;
    for (int64_t v = (int64_t)blockIdx.x * kWeighWaves + (threadIdx.x >> 6); v < units; v += (int64_t)gridDim.x * kWeighWaves) {
        const int64_t u = v / a.c.kv_heads;
        const int kv_head = (int)(v - u * a.c.kv_heads), seq = (int)(u / chunks), t0 = (int)(u - (int64_t)seq * chunks) * kPage;
        const int begin = a.c.q_start[seq], end = a.c.q_start[seq + 1];
        const int held = min(max(a.c.kv_len[seq], 0), (int)(a.c.max_pages * kPage));
        if (begin < 0 || end <= begin || end > a.N || t0 + place >= held) continue;
        const int id = a.c.table[seq * a.c.max_pages + t0 / kPage];
        if (id < 0 || id >= a.c.n_pages) continue;
        const int64_t at = ((int64_t)id * a.c.kv_heads + kv_head) * kPage + place;
        float sum = 0.0f;
#pragma unroll 4
        for (int i = 0; i < parts; ++i) sum += a.sums[(v * parts + i) * kPage + place];
        if (t0 + place < held - (end - begin) && a.decay != 0.0f) sum = fmaf(a.decay, a.old[at], sum);
        a.out[at] = sum;
    }
}

template <int D, bool BF16>
void launch_weigh_d(const WeighArgs &a, const WeighPlan &p, hipStream_t st) {
    constexpr int64_t kMost = 1 << 22;   // workgroups; more units take turns
    const int64_t stats = p.tiles * a.splits * a.c.kv_heads;
    hipLaunchKernelGGL((weigh_stats_kernel<D, BF16>), dim3((unsigned)std::min(stats, kMost)),
                       dim3(kWeighThreads), 0, st, a, stats);
    const int64_t pages = a.c.n_seqs * p.chunks * a.c.kv_heads, units = pages * p.parts;
    const dim3 g((unsigned)std::min(units, kMost));
    if (!p.many) {
        hipLaunchKernelGGL((weigh_few_kernel<D, BF16>), g, dim3(kWeighThreads), 0, st, a, p.chunks, units);
        return;
    }
    hipLaunchKernelGGL((weigh_many_kernel<D, BF16>), g, dim3(kWeighThreads), 0, st, a, p.chunks, p.parts, units);
    if (p.parts > 1)
        hipLaunchKernelGGL(weigh_join_kernel, dim3((unsigned)((pages + kWeighWaves - 1) / kWeighWaves)), dim3(kWeighThreads), 0,
                           st, a, p.chunks, p.parts, pages);
}

}  // namespace

hipError_t launch_kv4_weigh(const WeighArgs &a, const WeighPlan &p, int bf16, int dim, hipStream_t st) {
    if (dim == 64) { if (bf16) launch_weigh_d<64, true>(a, p, st); else launch_weigh_d<64, false>(a, p, st); }
    else if (dim == 128) { if (bf16) launch_weigh_d<128, true>(a, p, st); else launch_weigh_d<128, false>(a, p, st); }
    else { if (bf16) launch_weigh_d<256, true>(a, p, st); else launch_weigh_d<256, false>(a, p, st); }
    return hipGetLastError();
}

}  // namespace bitnet
