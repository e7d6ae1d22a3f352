// kv4_weigh.hip -- the attention weight that each token of the 4-bit cache gets from a call's
// rows, added to what it had got before: what an eviction goes by.
//
//   out[t] = (t older than the rows ? decay * old[t] : 0) + sum_r p_rt,
//   p_rt = 2^(x_rt - m_r) / sum_s 2^(x_rs - m_r),   x_rt = log2(e) * scale * q_r . k_t
// summed over the rows of a sequence and the heads that share a kv head, whose queries are
// rows of one problem as in attn_kv4.hip.
//
// Two launches.  The first gives each row's maximum m and sum, a workgroup to 16 rows and
// a share of the pages that they see, its waves taking turns at the pages.  The second has
// a wave to a page (or a workgroup, where there are many rows): it goes over the rows that
// see the page and keeps the page's 64 sums in registers, so no token is added to by two
// waves and the order of the sums is fixed.  Between them lie 8 bytes a row and share.
//
// q . k_t = sum_g step_tg (q_g . (code_tg - 8)) + mid_tg sum(q_g), the products of codes on
// the fp16 matrix instruction (q scaled by a power of two a row, in two fp16 terms of 22
// bits for fp32 rows, exactly for bf16 ones), all else in fp32.
#include <algorithm>

#include "codes4.h"
#include "kv4.h"

namespace bitnet {

namespace {

constexpr int kWeighThreads = 256;
constexpr int kWeighWaves = kWeighThreads / 64;

// A row's query: 8 channels of every 32 in this lane (quad), times 2^k; the sums of its
// groups at the same scale; and what makes a product of them a power of two's exponent.
template <int D, bool BF16>
struct Query {
    static constexpr int NT = BF16 ? 1 : 2, NS = D / 32, NG = D / 64;
    h8 f[NT][NS];
    float sum[NG], scale;
};
template <int D, bool BF16>
__device__ __forceinline__ void load_query(Query<D, BF16> &q, const void *p, int64_t at, float scale_log2) {
    using Q = Query<D, BF16>;
    float v[Q::NS][8], top = 0.0f;
#pragma unroll
    for (int j = 0; j < Q::NS; ++j) load8<BF16>(p, at + 32 * j, v[j]);
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

// A page's keys as they are loaded: this lane's codes of token 16 i + n, 8 channels of
// every 32, and the pairs of tokens 16 i + 4 quad + 0..3.
template <int D>
struct Keys {
    static constexpr int NS = D / 32, NG = D / 64;
    uint32_t code[4][NS], pair[4][4 * NG];
};
template <int D>
__device__ __forceinline__ void load_keys(Keys<D> &k, const uint8_t *rec, int n, int quad) {
    using L = Kv4Page<D>;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        load_words(rec + (16 * i + n) * L::kRow + quad * (D / 8), k.code[i]);
        const uint4 *p = reinterpret_cast<const uint4 *>(rec + L::kKeyPairs + (16 * i + 4 * quad) * L::kGroups * 4);
#pragma unroll
        for (int g = 0; g < L::kGroups; ++g) {
            const uint4 a = p[g];
            k.pair[i][4 * g] = a.x;
            k.pair[i][4 * g + 1] = a.y;
            k.pair[i][4 * g + 2] = a.z;
            k.pair[i][4 * g + 3] = a.w;
        }
    }
}
// x of token 16 i + 4 quad + e and this lane's row, in s[i][e].
template <int D, bool BF16>
__device__ __forceinline__ void scores(const Keys<D> &k, const Query<D, BF16> &q, uint32_t one,
                                       float (&s)[4][4]) {
    using Q = Query<D, BF16>;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f4 acc[Q::NG];
#pragma unroll
        for (int g = 0; g < Q::NG; ++g) {
            acc[g] = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int j = 2 * g; j < 2 * g + 2; ++j) {
                h2 c[4];
                codes8<false>(k.code[i][j], one, c);
                const h8 kc = join(c[0], c[1], c[2], c[3]);
#pragma unroll
                for (int t = 0; t < Q::NT; ++t) acc[g] = mfma(kc, q.f[t][j], acc[g]);
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float x = 0.0f;
#pragma unroll
            for (int g = 0; g < Q::NG; ++g) {
                const h2 p = as_h2(k.pair[i][e * Q::NG + g]);   // (step, middle)
                x = fmaf((float)p[0], acc[g][e], fmaf((float)p[1], q.sum[g], x));
            }
            s[i][e] = x * q.scale;
        }
    }
}

// Hides what a row at `pos`, whose window begins at `low`, does not see of page t0.
__device__ __forceinline__ void hide(float (&s)[4][4], int t0, int quad, int pos, int low, int sinks) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int j = t0 + 16 * i + 4 * quad + e;
            const bool hidden = (j > pos) | ((j < low) & (j >= sinks));
            s[i][e] = hidden ? -INFINITY : s[i][e];
        }
}

template <int D, bool BF16>
__global__ __launch_bounds__(kWeighThreads) void weigh_stats_kernel(const WeighArgs a, int64_t units) {
    using L = Kv4Page<D>;
    __shared__ float m_all[kWeighWaves][16], l_all[kWeighWaves][16];
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
        const uint32_t row = min(t.row0 + n, t.rows - 1), tok = row / G;
        const int head = kv_head * (int)G + (int)(row - tok * G);
        const int64_t line = (int64_t)(t.token0 + (int)tok) * a.heads + head;
        const int chunk = (t.pages + a.splits - 1) / a.splits;
        const int begin = min(split * chunk, t.pages), end = min(begin + chunk, t.pages);
        float m = kNoMax, l = 0.0f;
        if (begin < end) {
            Query<D, BF16> q;
            load_query(q, a.q, (t.token0 + (int64_t)tok) * a.q_stride + head * D + 8 * quad, a.scale_log2);
            const int pos = t.pos0 + (int)tok, low = a.window > 0 ? pos - a.window + 1 : 0;
            const int32_t *table = a.c.table + (int64_t)t.seq * a.c.max_pages;
            for (int from = begin + wave; from < end; from += 64 * kWeighWaves) {
                // 64 table entries of this wave at a time, one a lane
                const int i = from + kWeighWaves * lane;
                const int mine = i < end ? table[i < t.sink_pages ? i : t.first + i - t.sink_pages] : -1;
                uint64_t there = __ballot(mine >= 0 && mine < a.c.n_pages);
                while (there) {
                    const int bit = __builtin_ctzll(there);
                    there &= there - 1;
                    const int at = from + kWeighWaves * bit, id = __builtin_amdgcn_readlane(mine, bit);
                    const int t0 = (at < t.sink_pages ? at : t.first + at - t.sink_pages) * kPage;
                    Keys<D> k;
                    load_keys(k, a.c.cache + ((int64_t)id * a.c.kv_heads + kv_head) * L::kBytes, n, quad);
                    float s[4][4];
                    scores(k, q, one, s);
                    hide(s, t0, quad, pos, low, a.sinks);
                    float top = -INFINITY;
#pragma unroll
                    for (int i4 = 0; i4 < 4; ++i4)
#pragma unroll
                        for (int e = 0; e < 4; ++e) top = fmaxf(top, s[i4][e]);
                    const float m_new = fmaxf(m, top);
                    l *= __builtin_amdgcn_exp2f(m - m_new);
                    m = m_new;
#pragma unroll
                    for (int i4 = 0; i4 < 4; ++i4)
#pragma unroll
                        for (int e = 0; e < 4; ++e) l += __builtin_amdgcn_exp2f(s[i4][e] - m);
                }
            }
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
        if (threadIdx.x < 16 && t.row0 + n < t.rows) {
            float best = m_all[0][n], sum = 0.0f;
#pragma unroll
            for (int w = 1; w < kWeighWaves; ++w) best = fmaxf(best, m_all[w][n]);
#pragma unroll
            for (int w = 0; w < kWeighWaves; ++w)
                sum = fmaf(l_all[w][n], __builtin_amdgcn_exp2f(m_all[w][n] - best), sum);
            a.part[split * a.N * a.heads + line] = make_float2(best, sum);
        }
    }
}

// PAGES pages to a workgroup: one for each wave, or one whose rows the waves share.
template <int D, bool BF16, int PAGES>
__global__ __launch_bounds__(kWeighThreads) void weigh_pages_kernel(const WeighArgs a, int chunks,
                                                                    int64_t units) {
    using L = Kv4Page<D>;
    __shared__ float w_all[PAGES == 1 ? kWeighWaves : 1][64];
    const int lane = threadIdx.x & 63, n = lane & 15, quad = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t G = (uint32_t)a.heads / (uint32_t)a.c.kv_heads;
    const uint32_t one = ones_1024();
    constexpr uint32_t kTurns = PAGES == 1 ? kWeighWaves : 1;
    const uint32_t turn = PAGES == 1 ? wave : 0;
    for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const int64_t u = unit / a.c.kv_heads;
        const int kv_head = (int)(unit - u * a.c.kv_heads), seq = (int)(u / chunks), chunk = (int)(u - (int64_t)seq * chunks);
        const int begin = a.c.q_start[seq], end = a.c.q_start[seq + 1];
        const int64_t most = a.c.max_pages * kPage;
        const int held = min(max(a.c.kv_len[seq], 0), (int)most);
        if (begin < 0 || end <= begin || end > a.N) continue;   // the whole workgroup
        const int pos0 = held - (end - begin);
        const uint32_t rows = (uint32_t)(end - begin) * G;
        for (int first = chunk * PAGES; first * kPage < held; first += chunks * PAGES) {
            const int t0 = (first + (PAGES == 1 ? 0 : wave)) * kPage;
            const int id = t0 < held ? a.c.table[seq * a.c.max_pages + t0 / kPage] : -1;
            const bool there = id >= 0 && id < a.c.n_pages;
            float w[4][4] = {};
            if (there) {
                // the rows that see the page: from position t0 on, and not beyond the window
                uint32_t r0 = t0 > pos0 ? (uint32_t)(t0 - pos0) * G / 16 : 0, r1 = (rows + 15) / 16;
                if (a.window > 0 && t0 >= a.sinks) {
                    const int64_t last = (int64_t)t0 + kPage - 1 + a.window - 1 - pos0;   // the last token that does
                    r1 = last < 0 ? 0 : (uint32_t)min((int64_t)r1, ((last + 1) * G + 15) / 16);
                }
                Keys<D> k;
                if (r0 < r1)
                    load_keys(k, a.c.cache + ((int64_t)id * a.c.kv_heads + kv_head) * L::kBytes, n, quad);
                for (uint32_t r = r0 + turn; r < r1; r += kTurns) {
                    const uint32_t mine = r * 16 + n, row = min(mine, rows - 1), tok = row / G;
                    const int head = kv_head * (int)G + (int)(row - tok * G);
                    const int64_t line = (int64_t)(begin + (int)tok) * a.heads + head;
                    float2 ml = a.part[line];
                    for (int s = 1; s < a.splits; ++s) {
                        const float2 o = a.part[s * a.N * a.heads + line];
                        const float best = fmaxf(ml.x, o.x);
                        ml.y = ml.y * __builtin_amdgcn_exp2f(ml.x - best) + o.y * __builtin_amdgcn_exp2f(o.x - best);
                        ml.x = best;
                    }
                    Query<D, BF16> q;
                    load_query(q, a.q, (begin + (int64_t)tok) * a.q_stride + head * D + 8 * quad, a.scale_log2);
                    const int pos = pos0 + (int)tok, low = a.window > 0 ? pos - a.window + 1 : 0;
                    float x[4][4];
                    scores(k, q, one, x);
                    hide(x, t0, quad, pos, low, a.sinks);
                    // a row that sees nothing, or is no number, adds nothing; nor one behind the last
                    const bool good = ml.y > 0.0f && ml.y < INFINITY && mine < rows;
                    const float inv = good ? 1.0f / ml.y : 0.0f;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float p = __builtin_amdgcn_exp2f(x[i][e] - ml.x);
                            w[i][e] = good ? fmaf(p, inv, w[i][e]) : w[i][e];
                        }
                }
            }
            // over the 16 rows; lane n of a quad keeps token 16 (n / 4) + 4 quad + n % 4
            float mine = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float v = w[i][e];
                    v += dpp_f32<kDppXor1>(v);
                    v += dpp_f32<kDppXor2>(v);
                    v += dpp_f32<kDppHalfMirror>(v);
                    v += dpp_f32<kDppMirror>(v);
                    if (n == 4 * i + e) mine = v;
                }
            const int place = 16 * (n >> 2) + 4 * quad + (n & 3);
            if constexpr (PAGES == 1) {
                __syncthreads();
                w_all[wave][place] = mine;
                __syncthreads();
                mine = 0.0f;
                for (int k = 0; k < kWeighWaves; ++k) mine += w_all[k][place];
                if (wave != 0) continue;   // barriers are ahead of it for every wave
            }
            if (there && t0 + place < held) {
                const int64_t at = ((int64_t)id * a.c.kv_heads + kv_head) * kPage + place;
                if (t0 + place < pos0 && a.decay != 0.0f) mine = fmaf(a.decay, a.old[at], mine);
                a.out[at] = mine;
            }
        }
    }
}

template <int D, bool BF16>
void launch_weigh_d(const WeighArgs &a, const WeighPlan &p, hipStream_t st) {
    constexpr int64_t kMost = 1 << 22;   // workgroups; more units take turns
    const int64_t stats = p.tiles * a.splits * a.c.kv_heads;
    hipLaunchKernelGGL((weigh_stats_kernel<D, BF16>), dim3((unsigned)std::min(stats, kMost)),
                       dim3(kWeighThreads), 0, st, a, stats);
    const int64_t units = a.c.n_seqs * p.chunks * a.c.kv_heads;
    const dim3 g((unsigned)std::min(units, kMost));
    if (p.shared)
        hipLaunchKernelGGL((weigh_pages_kernel<D, BF16, 1>), g, dim3(kWeighThreads), 0, st, a, p.chunks, units);
    else
        hipLaunchKernelGGL((weigh_pages_kernel<D, BF16, kWeighWaves>), g, dim3(kWeighThreads), 0, st, a, p.chunks,
                           units);
}

}  // namespace

hipError_t launch_kv4_weigh(const WeighArgs &a, const WeighPlan &p, int bf16, int dim, hipStream_t st) {
    if (dim == 64) { if (bf16) launch_weigh_d<64, true>(a, p, st); else launch_weigh_d<64, false>(a, p, st); }
    else if (dim == 128) { if (bf16) launch_weigh_d<128, true>(a, p, st); else launch_weigh_d<128, false>(a, p, st); }
    else { if (bf16) launch_weigh_d<256, true>(a, p, st); else launch_weigh_d<256, false>(a, p, st); }
    return hipGetLastError();
}

}  // namespace bitnet
