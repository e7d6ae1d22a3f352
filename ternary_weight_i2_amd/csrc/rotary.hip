// rotary.hip -- rotary positions: rows turned to their positions, alone and on the
// way into the 4-bit cache.
//
// Pair i of a row at position p is turned by the angle 2 pi frac(p * turns_i / 2^64):
//   (a, b) -> (a c - b s, b c + a s),   c = fp32(magnitude cos), s = fp32(magnitude sin)
// with both products and their sum each rounded to fp32, and the result to the row's
// type.  turns_i is the frequency as a 64-bit fraction of a turn, so p * turns_i modulo
// 2^64 loses nothing however far p is, where an fp32 angle is off by 2^-24 p radians.
// The remainder of the nearest quarter turn, at most 1/8, goes through the Taylor series
// of sine and cosine in binary64 (off by less than 2^-52), so c and s are the nearest
// fp32 numbers to all but one in 2^27 and what is quantised of a key afterwards does
// not depend on how they were found.
//
// What bounds them: HBM for many rows (8191 of 32 heads of 80, bf16, 84 MB: 13.6 us where the
// last-level cache has a part of it; prompts of 6800 tokens, 16 + 8 heads of 128, with the
// append, 91 MB: 27 us, 3.4 TB/s), the launch and a chain of loads for few (64 rows of 32 heads
// 3.8 us; one token with the append 4.2).  Angles are found once for all heads of a
// workgroup's tokens and lie in LDS: 60 binary64 operations each, a few percent of a prompt.
#include <algorithm>

#include "kv4.h"

namespace bitnet {

namespace {

constexpr int kRotThreads = 256;
constexpr int kMaxPairs = 512;   // of a row: heads of up to 1024 channels

// c and s of a fraction of a turn.
__device__ __forceinline__ float2 cos_sin(uint64_t frac, double magnitude, double sign) {
    const uint64_t quarter = (frac + (1ull << 61)) >> 62;   // the nearest, 4 = 0
    const double x = (double)(int64_t)(frac - (quarter << 62)) * (6.283185307179586 / 0x1p64);
    const double z = x * x;
    double s = -1.0 / 1307674368000.0;           // -1/15!, up to x^15
    s = fma(s, z, 1.0 / 6227020800.0);
    s = fma(s, z, -1.0 / 39916800.0);
    s = fma(s, z, 1.0 / 362880.0);
    s = fma(s, z, -1.0 / 5040.0);
    s = fma(s, z, 1.0 / 120.0);
    s = fma(s, z, -1.0 / 6.0);
    s = fma(s * z, x, x);
    double c = 1.0 / 20922789888000.0;           // 1/16!, up to x^16
    c = fma(c, z, -1.0 / 87178291200.0);
    c = fma(c, z, 1.0 / 479001600.0);
    c = fma(c, z, -1.0 / 3628800.0);
    c = fma(c, z, 1.0 / 40320.0);
    c = fma(c, z, -1.0 / 720.0);
    c = fma(c, z, 1.0 / 24.0);
    c = fma(c, z, -0.5);
    c = fma(c, z, 1.0);
    const bool swap = quarter & 1;
    double co = swap ? s : c, si = swap ? c : s;
    if (quarter == 1 || quarter == 2) co = -co;
    if (quarter == 2 || quarter == 3) si = -si;
    return make_float2((float)(magnitude * co), (float)(sign * magnitude * si));
}

__device__ __forceinline__ float2 turned(float a, float b, float2 cs) {
#pragma clang fp contract(off)
    const float ac = a * cs.x, bs = b * cs.y, bc = b * cs.x, as = a * cs.y;
    return make_float2(ac - bs, bc + as);
}

template <bool BF16>
__device__ __forceinline__ void put1(void *p, int64_t i, float v) {
    if constexpr (BF16) static_cast<uint16_t *>(p)[i] = (uint16_t)bf16_bits(v);
    else static_cast<float *>(p)[i] = v;
}

// How a row is cut into a thread's items.  kHalves: eight pairs (i, i + rot/2), read and
// written as two runs of eight channels, rot a multiple of 16; kNeighbours: eight
// channels, pairs (2 i, 2 i + 1); kSingle: one pair (i, i + rot/2) of any even rot.  What
// lies behind the first rot channels is copied, by items of its own.
enum Cut { kHalves, kNeighbours, kSingle };
__host__ __device__ constexpr int items_of(Cut cut, int dim, int rot) {
    return cut == kHalves ? rot / 16 + (dim - rot) / 8
           : cut == kNeighbours ? dim / 8
                                : rot / 2 + (dim - rot);
}
Cut cut_of(const RotaryArgs &r) {
    return r.interleaved ? kNeighbours : r.rot % 16 ? kSingle : kHalves;
}

// Item j of a head's row, at x (out may be x: nothing else reads what an item writes).
template <Cut CUT, bool BF16>
__device__ __forceinline__ void turn_item(const void *x, int64_t xi, void *out, int64_t oi, int j,
                                          int rot, const float2 *cs) {
    if constexpr (CUT == kHalves) {
        if (j < rot / 16) {
            float a[8], b[8];
            load8<BF16>(x, xi + 8 * j, a);
            load8<BF16>(x, xi + rot / 2 + 8 * j, b);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float2 t = turned(a[e], b[e], cs[8 * j + e]);
                a[e] = t.x;
                b[e] = t.y;
            }
            store8_values<BF16>(out, oi + 8 * j, a);
            store8_values<BF16>(out, oi + rot / 2 + 8 * j, b);
        } else {
            const int ch = rot + 8 * (j - rot / 16);
            float a[8];
            load8<BF16>(x, xi + ch, a);
            store8_values<BF16>(out, oi + ch, a);
        }
    } else if constexpr (CUT == kNeighbours) {
        float a[8];
        load8<BF16>(x, xi + 8 * j, a);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            if (8 * j + e >= rot) continue;
            const float2 t = turned(a[e], a[e + 1], cs[4 * j + e / 2]);
            a[e] = t.x;
            a[e + 1] = t.y;
        }
        store8_values<BF16>(out, oi + 8 * j, a);
    } else {
        const int h = rot / 2;
        if (j < h) {
            const float2 t = turned(load1<BF16>(x, xi + j), load1<BF16>(x, xi + h + j), cs[j]);
            put1<BF16>(out, oi + j, t.x);
            put1<BF16>(out, oi + h + j, t.y);
        } else {
            put1<BF16>(out, oi + h + j, load1<BF16>(x, xi + h + j));
        }
    }
}

// `tokens` rows of heads * dim from blockIdx.x * tokens on, a share of their items.
template <Cut CUT, bool BF16>
__global__ __launch_bounds__(kRotThreads) void rotary_kernel(
    const RotaryArgs r, const void *x, int64_t x_stride, void *out, int64_t out_stride, int64_t N,
    int heads, int dim, int tokens, const int32_t *positions) {
    extern __shared__ float2 cs[];   // [tokens][rot / 2]
    const int64_t first = (int64_t)blockIdx.x * tokens;
    const int mine = (int)min((int64_t)tokens, N - first), half = r.rot / 2;
    for (int i = threadIdx.x; i < mine * half; i += kRotThreads) {
        const int t = i / half, f = i - t * half;
        cs[i] = cos_sin((uint64_t)((int64_t)positions[first + t]) * (uint64_t)r.turns[f], r.magnitude, r.sign);
    }
    __syncthreads();
    const int items = items_of(CUT, dim, r.rot), row = items * heads;
    for (int i = blockIdx.y * kRotThreads + threadIdx.x; i < mine * row; i += kRotThreads * gridDim.y) {
        const int t = i / row, in_row = i - t * row, head = in_row / items, j = in_row - head * items;
        turn_item<CUT, BF16>(x, (first + t) * x_stride + head * dim, out,
                             (first + t) * out_stride + head * dim, j, r.rot, cs + t * half);
    }
}

struct AppendRows {
    const void *q, *k, *v;
    void *q_out;
    int64_t q_stride, out_stride, k_stride, v_stride;
    const int32_t *offset;
    int heads;
};

// kv4_append_kernel (kv4.hip) with the keys turned first, and the queries of the same
// four tokens turned beside them.
template <int D, Cut CUT, bool BF16>
__global__ __launch_bounds__(kRotThreads) void rotary_append_kernel(const RotaryArgs r, const Kv4Args c,
                                                                    const AppendRows a, int64_t N) {
    using L = Kv4Page<D>;
    __shared__ float2 cs[4 * D / 2];   // [token][rot / 2]
    const Block4 at = find_block(c, N);
    if (!at.rows) return;   // the whole workgroup
    const int half = r.rot / 2, t0 = at.in_page;
    const int64_t pos = (int64_t)at.base + (a.offset ? a.offset[at.seq] : 0);
    for (int i = threadIdx.x; i < 4 * half; i += kRotThreads) {
        const int t = i / half, f = i - t * half;
        if (at.rows >> t & 1)
            cs[i] = cos_sin((uint64_t)(pos + t) * (uint64_t)r.turns[f], r.magnitude, r.sign);
    }
    __syncthreads();
    const int kv_lanes = c.kv_heads * 2 * (D / 8), items = items_of(CUT, D, r.rot);
    const int lanes = kv_lanes + a.heads * items;
    for (int i = blockIdx.y * kRotThreads + threadIdx.x; i < lanes; i += kRotThreads * gridDim.y) {
        if (i >= kv_lanes) {   // a query item, of all four tokens
            const int head = (i - kv_lanes) / items, j = i - kv_lanes - head * items;
#pragma unroll
            for (int t = 0; t < 4; ++t)
                if (at.rows >> t & 1)
                    turn_item<CUT, BF16>(a.q, (at.row + t) * a.q_stride + head * D, a.q_out,
                                         (at.row + t) * a.out_stride + head * D, j, r.rot,
                                         cs + t * half);
            continue;
        }
        // eight channels of a key or a value, of all four tokens: whole groups of eight lanes
        const int p = i % (D / 8), head = i / (D / 8) >> 1;
        const bool is_v = i / (D / 8) & 1;
        uint32_t codes[4], pair[4];
        float x[4][8];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            if (!(at.rows >> t & 1)) continue;
            const int64_t n = at.row + t;
            if (is_v) {
                load8<BF16>(a.v, n * a.v_stride + head * D + 8 * p, x[t]);
                continue;
            }
            const int64_t xi = n * a.k_stride + head * D;
            load8<BF16>(a.k, xi + 8 * p, x[t]);
            const float2 *const ct = cs + t * half;
            if constexpr (CUT == kNeighbours) {
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    if (8 * p + e >= r.rot) continue;
                    const float2 o = turned(x[t][e], x[t][e + 1], ct[4 * p + e / 2]);
                    x[t][e] = o.x;
                    x[t][e + 1] = o.y;
                }
            } else if constexpr (CUT == kHalves) {
                if (8 * p < r.rot) {
                    const bool lower = 8 * p < half;
                    float y[8];
                    load8<BF16>(a.k, xi + 8 * p + (lower ? half : -half), y);
                    const float2 *const cp = ct + 8 * p - (lower ? 0 : half);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        x[t][e] = lower ? turned(x[t][e], y[e], cp[e]).x : turned(y[e], x[t][e], cp[e]).y;
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int ch = 8 * p + e;
                    if (ch >= r.rot) continue;
                    const bool lower = ch < half;
                    const float y = load1<BF16>(a.k, xi + (lower ? ch + half : ch - half));
                    const float2 f = ct[lower ? ch : ch - half];
                    x[t][e] = lower ? turned(x[t][e], y, f).x : turned(y, x[t][e], f).y;
                }
            }
            if constexpr (BF16)   // as the turned rows are stored
#pragma unroll
                for (int e = 0; e < 8; ++e) x[t][e] = __uint_as_float(bf16_bits(x[t][e]) << 16);
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) codes[t] = quantise8(x[t], &pair[t]);
        if (!at.cached(c)) continue;   // the queries are still to be turned
        uint8_t *rec = c.cache + ((int64_t)at.page * c.kv_heads + head) * L::kBytes;
        store_block4<D>(rec, is_v, t0, p, at.rows, codes, pair);
    }
}

template <int D, Cut CUT>
void launch_append_d(const RotaryArgs &r, const Kv4Args &c, const AppendRows &a, int bf16, int64_t N,
                     hipStream_t st) {
    // A workgroup's sequence, angles and rows are a chain of loads, so the lanes of few
    // tokens are spread over several; a prompt's blocks keep theirs together, which shares
    // the angles, unless there are very many (16 heads of 256, pairs of single channels: 45.8 us
    // whole, 37.6 in two; 8 + 16 heads of 128, 64 to 384 threads in 1 to 6: 38 to 44 us, 39 so).
    const int lanes = c.kv_heads * 2 * (D / 8) + a.heads * items_of(CUT, D, r.rot);
    const int64_t blocks = N / 4 + 2 * c.n_seqs;
    const int turns = (lanes + kRotThreads - 1) / kRotThreads, spread = blocks <= 256 ? turns : turns > 4 ? 2 : 1;
    const dim3 g((unsigned)blocks, (unsigned)spread), t(kRotThreads);
    if (bf16) hipLaunchKernelGGL((rotary_append_kernel<D, CUT, true>), g, t, 0, st, r, c, a, N);
    else hipLaunchKernelGGL((rotary_append_kernel<D, CUT, false>), g, t, 0, st, r, c, a, N);
}

template <int D>
void launch_append(const RotaryArgs &r, const Kv4Args &c, const AppendRows &a, int bf16, int64_t N,
                   hipStream_t st) {
    const Cut cut = cut_of(r);
    if (cut == kHalves) launch_append_d<D, kHalves>(r, c, a, bf16, N, st);
    else if (cut == kNeighbours) launch_append_d<D, kNeighbours>(r, c, a, bf16, N, st);
    else launch_append_d<D, kSingle>(r, c, a, bf16, N, st);
}

}  // namespace

hipError_t launch_rotary(const RotaryArgs &r, const void *x, int64_t x_stride, void *out,
                         int64_t out_stride, int bf16, int64_t N, int heads, int dim,
                         const int32_t *positions, hipStream_t st) {
    const Cut cut = cut_of(r);
    const int row = items_of(cut, dim, r.rot) * heads;
    // about two items to a thread; a row of many is spread over workgroups
    const int per = 2 * kRotThreads;
    const int tokens = row >= per ? 1 : std::min(per / row, kMaxPairs * 4 / (r.rot / 2));
    const int spread = row >= per ? (row + per - 1) / per : 1;
    const dim3 g((unsigned)((N + tokens - 1) / tokens), (unsigned)spread), t(kRotThreads);
    const size_t lds = (size_t)tokens * (r.rot / 2) * sizeof(float2);
#define ROTARY(C, B)                                                                             \
    hipLaunchKernelGGL((rotary_kernel<C, B>), g, t, lds, st, r, x, x_stride, out, out_stride, N, \
                       heads, dim, tokens, positions)
    if (cut == kHalves) { if (bf16) ROTARY(kHalves, true); else ROTARY(kHalves, false); }
    else if (cut == kNeighbours) { if (bf16) ROTARY(kNeighbours, true); else ROTARY(kNeighbours, false); }
    else { if (bf16) ROTARY(kSingle, true); else ROTARY(kSingle, false); }
#undef ROTARY
    return hipGetLastError();
}

hipError_t launch_rotary_append(const RotaryArgs &r, const Kv4Args &c, const void *q,
                                int64_t q_stride, void *q_out, int64_t out_stride, int heads,
                                const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                                const int32_t *offset, int bf16, int64_t N, int dim,
                                hipStream_t st) {
    const AppendRows a{q, k, v, q_out, q_stride, out_stride, k_stride, v_stride, offset, heads};
    if (dim == 64) launch_append<64>(r, c, a, bf16, N, st);
    else if (dim == 128) launch_append<128>(r, c, a, bf16, N, st);
    else launch_append<256>(r, c, a, bf16, N, st);
    return hipGetLastError();
}

}  // namespace bitnet
