// w4.hip -- matrices of 4-bit weights with a step for each group of channels: the
// quantiser, rows back as floats, and the product with float tokens.
//
//   weight = step * (code - 8),   step fp16, one for each row and GROUP channels
//   y[n][m] = sum_g step_mg * sum_{k in g} x_nk (code_mk - 8)
//
// Layout: tiles of 16 rows, blocks of 128 channels.  codes[tile][block][quad][row][j] is a
// dword with channels 32 j + 8 quad + 0..7 of the block, the first in its low bits: 16
// bytes of a lane (quad, row), 1 KB side by side for a wave, and each dword one operand
// of the 16x16x32 matrix instruction.  steps[tile][block][row][128 / GROUP].
//
// The product runs on that instruction for any number of tokens: a code becomes code - 8 in
// fp16 exactly, a token's 128 channels are scaled by a power of two so that the largest is
// in [2^14, 2^15) and carried in one fp16 term (bf16 tokens: exact down to 2^-39 of the
// block's largest) or two (fp32: 22 bits, no finer than 2^-40 of the largest).  A group's sum and
// the sum over groups are fp32.
#include <algorithm>

#include "codes4.h"
#include "layer.h"

namespace bitnet {

namespace {

constexpr int kW4Threads = 512;
constexpr int kW4Waves = kW4Threads / 64;
constexpr int kAhead = 4;                 // blocks of 1 KB that a wave has on the way
constexpr float kW4Max = 7.0f * 65504.0f; // 7 steps of the largest fp16

// ---------------------------------------------------------------- quantiser

// A wave takes a tile's block: lane (row, quad), 8 channels of each 32.  FORM 0: fp32, 1:
// bf16 weights; 2: int8 codes -8..7 with steps given as [M][K / GROUP].
template <int FORM, int GS>
__global__ __launch_bounds__(256) void w4_pack_kernel(const void *w, const uint16_t *given, int64_t M,
                                                      int64_t K, uint8_t *codes, uint16_t *steps) {
#pragma clang fp contract(off)
    const int lane = threadIdx.x & 63, row = lane & 15, quad = lane >> 4;
    const int64_t nblk = K / 128, m = (int64_t)blockIdx.x * 16 + row;
    for (int64_t blk = blockIdx.y * 4 + (threadIdx.x >> 6); blk < nblk; blk += 4 * gridDim.y) {
        const int64_t at = m * K + blk * 128 + 8 * quad, out = ((int64_t)blockIdx.x * nblk + blk) * 64 + lane;
        uint32_t word[4] = {0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u};
        uint16_t st[GS] = {};
        if constexpr (FORM == 2) {
            if (m < M) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint2 b = *reinterpret_cast<const uint2 *>(static_cast<const int8_t *>(w) + at + 32 * j);
                    word[j] = 0;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int c = (int8_t)((e < 4 ? b.x : b.y) >> (8 * (e & 3)));
                        word[j] |= (uint32_t)(min(max(c, -8), 7) + 8) << (4 * e);
                    }
                }
#pragma unroll
                for (int g = 0; g < GS; ++g) st[g] = given[(m * nblk + blk) * GS + g];
            }
        } else {
            float x[4][8];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (m < M) load8<FORM == 1>(w, at + 32 * j, x[j]);
                else
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[j][e] = 0.0f;
#pragma unroll
            for (int g = 0; g < GS; ++g) {
                constexpr int JS = 4 / GS;   // of the four runs of 32 channels
                float lo = kW4Max, hi = -kW4Max;
#pragma unroll
                for (int j = g * JS; j < (g + 1) * JS; ++j)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float v = x[j][e] == x[j][e] ? x[j][e] : 0.0f;
                        x[j][e] = __builtin_amdgcn_fmed3f(v, -kW4Max, kW4Max);
                        lo = fminf(lo, x[j][e]);
                        hi = fmaxf(hi, x[j][e]);
                    }
                for (int d = 16; d < 64; d *= 2) {
                    lo = fminf(lo, __shfl_xor(lo, d));
                    hi = fmaxf(hi, __shfl_xor(hi, d));
                }
                const _Float16 s16 = (_Float16)fmaxf(hi * (1.0f / 7.0f), lo * -0.125f);
                const float s = (float)s16, inv = s > 0.0f ? 1.0f / s : 0.0f;
                st[g] = __builtin_bit_cast(uint16_t, s16);
#pragma unroll
                for (int j = g * JS; j < (g + 1) * JS; ++j) {
                    word[j] = 0;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float c = __builtin_amdgcn_fmed3f(rintf(x[j][e] * inv), -8.0f, 7.0f);
                        word[j] |= (uint32_t)((int)c + 8) << (4 * e);
                    }
                }
            }
        }
        reinterpret_cast<uint4 *>(codes)[out] = make_uint4(word[0], word[1], word[2], word[3]);
        if (quad == 0)
#pragma unroll
            for (int g = 0; g < GS; ++g)
                steps[(((int64_t)blockIdx.x * nblk + blk) * 16 + row) * GS + g] = st[g];
    }
}

// Row ids[i] (or i) as floats, zeros where there is no such row.
template <bool BF16>
__global__ __launch_bounds__(256) void w4_rows_kernel(const W4Args w, const int32_t *ids, void *out) {
#pragma clang fp contract(off)
    const int64_t i = blockIdx.x, nblk = w.K / 128;
    const int64_t m = ids ? ids[i] : i;
    const bool there = m >= 0 && m < w.M;
    for (int p = threadIdx.x; p < w.K / 8; p += 256) {   // 8 channels: block, j, quad
        const int blk = p >> 4, j = p >> 2 & 3, quad = p & 3;
        uint32_t c = 0;
        float s = 0.0f;
        if (there) {
            const int64_t at = (m >> 4) * nblk + blk;
            c = reinterpret_cast<const uint32_t *>(w.codes)[(at * 64 + quad * 16 + (m & 15)) * 4 + j];
            s = (float)__builtin_bit_cast(
                _Float16, w.steps[(at * 16 + (m & 15)) * w.groups + (w.groups == 4 ? j : w.groups == 2 ? j >> 1 : 0)]);
        }
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = there ? s * (float)((int)(c >> (4 * e) & 15u) - 8) : 0.0f;
        store8_values<BF16>(out, i * w.K + 8 * p, x);
    }
}

// ---------------------------------------------------------------- product

// 128 channels of a token as the instruction takes them: 16 lanes with 8 channels each.
// The lane's eight as fp16 in the order of codes8, and what the scale has to be undone by.
template <int NT>
__device__ __forceinline__ float halves_of(const float (&x)[8], h8 (&t)[NT]) {
    float top = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(x[e]));
    top = fmaxf(top, dpp_f32<kDppXor1>(top));
    top = fmaxf(top, dpp_f32<kDppXor2>(top));
    top = fmaxf(top, dpp_f32<kDppHalfMirror>(top));
    top = fmaxf(top, dpp_f32<kDppMirror>(top));
    const int k = top > 0.0f ? min(15 - __builtin_amdgcn_frexp_expf(top), 126) : 0;
    const float up = ldexpf(1.0f, k);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float z = x[(e >> 1) + 4 * (e & 1)] * up;
        const _Float16 hi = (_Float16)z;
        t[0][e] = hi;
        if constexpr (NT == 2) t[1][e] = (_Float16)(z - (float)hi);
    }
    return ldexpf(1.0f, -k);
}

template <int GS>
struct StepWord;
template <> struct StepWord<1> { using type = uint16_t; };
template <> struct StepWord<2> { using type = uint32_t; };
template <> struct StepWord<4> { using type = uint2; };
__device__ __forceinline__ float step_of(uint16_t w, int) {
    return (float)__builtin_bit_cast(_Float16, w);
}
__device__ __forceinline__ float step_of(uint32_t w, int g) { return (float)as_h2(w)[g]; }
__device__ __forceinline__ float step_of(const uint2 &w, int g) {
    return (float)as_h2(g < 2 ? w.x : w.y)[g & 1];
}

// The tokens of blockIdx.y (up to 16 * TT) times tiles of rows.  WK of a workgroup's eight
// waves share a tile's blocks; the others have tiles of their own, every gridDim.x * 8 / WK
// on.  The tokens lie in LDS as operands: all of their channels if they fit, else `chunk`
// blocks at a time.
template <bool BF16, int TT, int GS>
__global__ __launch_bounds__(kW4Threads) void w4_linear_kernel(const W4Args w, const void *x, int64_t N,
                                                               float *y, int wk, int chunk, int iters) {
    constexpr int NT = BF16 ? 1 : 2;
    extern __shared__ __align__(16) uint8_t lds[];
    const int lane = threadIdx.x & 63, n = lane & 15, quad = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t tok0 = (int64_t)blockIdx.y * 16 * TT;
    const int toks = (int)min(N - tok0, (int64_t)(16 * TT));
    const int nblk = w.K / 128, tiles = (w.M + 15) / 16;
    h8 *const xs = reinterpret_cast<h8 *>(lds);            // [block][j][term][quad][token]
    float *const sc = reinterpret_cast<float *>(lds + (size_t)chunk * 256 * NT * toks);   // [block][16 TT]
    float4 *const red = reinterpret_cast<float4 *>(sc + chunk * 16 * TT);                 // [wave][TT][lane]

    // ---- this wave's blocks: shares of the chunks, tile by tile
    const int part = wave % wk, slot = wave / wk, slots = kW4Waves / wk;
    const int chunks = (nblk + chunk - 1) / chunk;
    auto tile_at = [&](int it) { return ((int)blockIdx.x + it * (int)gridDim.x) * slots + slot; };
    struct Run { int tile, from, to; };
    auto run_at = [&](int it, int c) {
        const int b0 = c * chunk, cnt = min(chunk, nblk - b0);
        return Run{min(tile_at(it), tiles - 1), b0 + cnt * part / wk, b0 + cnt * (part + 1) / wk};
    };
    using Word = typename StepWord<GS>::type;
    uint4 raw[kAhead];
    Word st[kAhead];
    auto load = [&](int u, const Run &r, int blk) {
        const int64_t at = (int64_t)r.tile * nblk + min(blk, nblk - 1);
        raw[u] = reinterpret_cast<const uint4 *>(w.codes)[at * 64 + lane];
        st[u] = reinterpret_cast<const Word *>(w.steps)[at * 16 + n];
    };
    auto after = [&](int it, int c) {   // the run that follows, or the same at the end
        if (c + 1 < chunks) return run_at(it, c + 1);
        return it + 1 < iters ? run_at(it + 1, 0) : run_at(it, c);
    };
    Run now = run_at(0, 0);
    {
        const Run next = after(0, 0);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const bool here = now.from + u < now.to;
            load(u, here ? now : next, here ? now.from + u : next.from + u);
        }
    }
    const uint32_t one = ones_1024();

    auto stage = [&](int c) {
        const int b0 = c * chunk, cnt = min(chunk, nblk - b0), p = threadIdx.x & 15;
        const int units = cnt * toks;   // (block, token): 16 lanes with 8 channels each
        constexpr int kBatch = 4, kStep = kW4Threads / 16;
        for (int u0 = threadIdx.x >> 4; u0 < units; u0 += kBatch * kStep) {
            float v[kBatch][8];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int u = min(u0 + i * kStep, units - 1), blk = u / toks, t = u - blk * toks;
                load8<BF16>(x, (tok0 + t) * w.K + (b0 + blk) * 128 + 8 * p, v[i]);
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int u = u0 + i * kStep;
                if (u >= units) break;   // the same for the 16 lanes
                const int blk = u / toks, t = u - blk * toks;
                h8 h[NT];
                const float down = halves_of<NT>(v[i], h);
#pragma unroll
                for (int k = 0; k < NT; ++k)
                    xs[(((blk * 4 + (p >> 2)) * NT + k) * 4 + (p & 3)) * toks + t] = h[k];
                if (p == 0) sc[blk * 16 * TT + t] = down;
            }
        }
    };
    if (chunks == 1) {
        stage(0);
        __syncthreads();
    }
    int tok[TT];   // the operand's token of this lane: those behind the last are repeated
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) tok[tt] = min(16 * tt + n, toks - 1);

    for (int it = 0; it < iters; ++it) {
        f4 sum[TT];
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) sum[tt] = f4{0.0f, 0.0f, 0.0f, 0.0f};
        for (int c = 0; c < chunks; ++c) {
            if (chunks > 1) {
                __syncthreads();
                stage(c);
                __syncthreads();
            }
            now = run_at(it, c);
            const Run next = after(it, c);
            for (int b = now.from; b < now.to; b += kAhead) {
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    if (b + u >= now.to) continue;   // the slot holds the next run's block
                    const int lb = b + u - c * chunk;
                    const h8 *const xb = xs + lb * 16 * NT * toks + quad * toks;
                    f4 s[TT];
#pragma unroll
                    for (int tt = 0; tt < TT; ++tt)
                        s[tt] = *reinterpret_cast<const f4 *>(sc + (lb * TT + tt) * 16 + 4 * quad);
                    const uint32_t word[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
                    f4 block[TT];
#pragma unroll
                    for (int g = 0; g < GS; ++g) {
                        f4 acc[TT];
#pragma unroll
                        for (int tt = 0; tt < TT; ++tt) acc[tt] = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                        for (int j = g * 4 / GS; j < (g + 1) * 4 / GS; ++j) {
                            h2 q[4];
                            codes8<false>(word[j], one, q);
                            const h8 wq = join(q[0], q[1], q[2], q[3]);
#pragma unroll
                            for (int tt = 0; tt < TT; ++tt)
#pragma unroll
                                for (int k = 0; k < NT; ++k)
                                    acc[tt] = mfma(xb[(j * NT + k) * 4 * toks + tok[tt]], wq, acc[tt]);
                        }
                        const float step = step_of(st[u], g);
#pragma unroll
                        for (int tt = 0; tt < TT; ++tt)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                block[tt][e] = g == 0 ? acc[tt][e] * step : fmaf(acc[tt][e], step, block[tt][e]);
                    }
#pragma unroll
                    for (int tt = 0; tt < TT; ++tt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) sum[tt][e] = fmaf(block[tt][e], s[tt][e], sum[tt][e]);
                    const bool here = b + u + kAhead < now.to;
                    load(u, here ? now : next, here ? b + u + kAhead : next.from + u);
                }
            }
            // slots that a short run had no block for
            if (now.to - now.from < kAhead)
#pragma unroll
                for (int u = 0; u < kAhead; ++u)
                    if (now.from + u >= now.to) load(u, next, next.from + u);
        }
        // ---- the tile's rows: lane (n, quad) has row n of tokens 4 quad + e
        const int tile = tile_at(it), m = tile * 16 + n;
        if (wk > 1) {
            __syncthreads();
#pragma unroll
            for (int tt = 0; tt < TT; ++tt)
                red[(wave * TT + tt) * 64 + lane] = make_float4(sum[tt][0], sum[tt][1], sum[tt][2], sum[tt][3]);
            __syncthreads();
            if (part == 0)
#pragma unroll
                for (int tt = 0; tt < TT; ++tt)
                    for (int k = 1; k < wk; ++k) {
                        const float4 o = red[((wave + k) * TT + tt) * 64 + lane];
                        sum[tt][0] += o.x;
                        sum[tt][1] += o.y;
                        sum[tt][2] += o.z;
                        sum[tt][3] += o.w;
                    }
        }
        if (part == 0 && m < w.M)
#pragma unroll
            for (int tt = 0; tt < TT; ++tt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int t = 16 * tt + 4 * quad + e;
                    if (t < toks) y[(tok0 + t) * w.M + m] = sum[tt][e];
                }
    }
}

// More tokens than 16: a workgroup has 16 * TT tokens and eight waves of RT tiles each, over
// a share of the blocks (blockIdx.z).  The tokens' operands are made `CB` blocks at a time in
// one half of the LDS while the matrix instructions read the other half: the values for it
// are on their way meanwhile, and so is each block of weights a turn ahead of its use.
// Token t of the 16 bytes (j, quad) = p lies in slot (t + 4 p) mod 16 TT, so that the lanes
// that write eight channels each of a few tokens spread over all banks.
template <bool BF16, int TT, int GS, int RT>
__global__ __launch_bounds__(kW4Threads, 2) void w4_wide_kernel(const W4Args w, const void *x, int64_t N,
                                                                float *y, float *part) {
    constexpr int NT = BF16 ? 1 : 2, CB = 4 / NT, TOK = 16 * TT;
    constexpr int kPieces = CB * TOK * 16 / kW4Threads;   // of 8 channels, for a thread
    __shared__ h8 xs[2][CB * 16 * NT][TOK];
    __shared__ __align__(16) float sc[2][CB][TOK];
    const int lane = threadIdx.x & 63, n = lane & 15, quad = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t tok0 = (int64_t)blockIdx.y * TOK;
    const int toks = (int)min(N - tok0, (int64_t)TOK);
    const int nblk = w.K / 128, tiles = (w.M + 15) / 16;
    const int begin = (int)((int64_t)nblk * blockIdx.z / gridDim.z), end = (int)((int64_t)nblk * (blockIdx.z + 1) / gridDim.z);
    const int tile0 = ((int)blockIdx.x * kW4Waves + wave) * RT;
    using Word = typename StepWord<GS>::type;
    uint4 raw[CB][RT];
    Word st[CB][RT];
    auto load_weights = [&](int c, int blk) {
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const int64_t at = (int64_t)min(tile0 + r, tiles - 1) * nblk + min(blk, end - 1);
            raw[c][r] = reinterpret_cast<const uint4 *>(w.codes)[at * 64 + lane];
            st[c][r] = reinterpret_cast<const Word *>(w.steps)[at * 16 + n];
        }
    };
    float v[kPieces][8];
    const int p = threadIdx.x & 15, u0 = threadIdx.x >> 4;   // piece i: unit u0 + 32 i, a token's block
    auto load_tokens = [&](int b0) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int u = u0 + 32 * i, blk = min(b0 + u / TOK, end - 1), t = min(u % TOK, toks - 1);
            load8<BF16>(x, (tok0 + t) * w.K + (int64_t)blk * 128 + 8 * p, v[i]);
        }
    };
    auto put_tokens = [&](int half) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int u = u0 + 32 * i, blk = u / TOK, t = u % TOK;
            h8 h[NT];
            const float down = halves_of<NT>(v[i], h);
#pragma unroll
            for (int k = 0; k < NT; ++k) xs[half][(blk * 4 + (p >> 2)) * NT * 4 + k * 4 + (p & 3)][(t + 4 * p) % TOK] = h[k];
            if (p == 0) sc[half][blk][t] = down;
        }
    };
    load_tokens(begin);
#pragma unroll
    for (int c = 0; c < CB; ++c) load_weights(c, begin + c);
    put_tokens(0);
    __syncthreads();
    const uint32_t one = ones_1024();
    f4 sum[RT][TT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) sum[r][tt] = f4{0.0f, 0.0f, 0.0f, 0.0f};
    int half = 0;
    for (int b0 = begin; b0 < end; b0 += CB, half ^= 1) {
        const bool more = b0 + CB < end;
        if (more) load_tokens(b0 + CB);
#pragma unroll
        for (int c = 0; c < CB; ++c) {
            if (b0 + c >= end) continue;
            f4 block[RT][TT];
#pragma unroll
            for (int g = 0; g < GS; ++g) {
                f4 acc[RT][TT];
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int tt = 0; tt < TT; ++tt) acc[r][tt] = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int j = g * 4 / GS; j < (g + 1) * 4 / GS; ++j) {
                    h8 wq[RT];
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        const uint32_t word = j == 0 ? raw[c][r].x : j == 1 ? raw[c][r].y : j == 2 ? raw[c][r].z : raw[c][r].w;
                        h2 q[4];
                        codes8<false>(word, one, q);
                        wq[r] = join(q[0], q[1], q[2], q[3]);
                    }
#pragma unroll
                    for (int tt = 0; tt < TT; ++tt)
#pragma unroll
                        for (int k = 0; k < NT; ++k) {
                            const h8 a = xs[half][(c * 4 + j) * NT * 4 + k * 4 + quad][(16 * tt + n + 4 * (4 * j + quad)) % TOK];
#pragma unroll
                            for (int r = 0; r < RT; ++r) acc[r][tt] = mfma(a, wq[r], acc[r][tt]);
                        }
                }
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const float step = step_of(st[c][r], g);
#pragma unroll
                    for (int tt = 0; tt < TT; ++tt)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            block[r][tt][e] = g == 0 ? acc[r][tt][e] * step : fmaf(acc[r][tt][e], step, block[r][tt][e]);
                }
            }
#pragma unroll
            for (int tt = 0; tt < TT; ++tt) {
                const f4 s = *reinterpret_cast<const f4 *>(&sc[half][c][16 * tt + 4 * quad]);
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sum[r][tt][e] = fmaf(block[r][tt][e], s[e], sum[r][tt][e]);
            }
            load_weights(c, b0 + c + CB);
        }
        if (more) put_tokens(half ^ 1);
        __syncthreads();
    }
    float *const out = gridDim.z > 1 ? part + (int64_t)blockIdx.z * N * w.M : y;
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int m = (tile0 + r) * 16 + n;
        if (m < w.M)
#pragma unroll
            for (int tt = 0; tt < TT; ++tt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int t = 16 * tt + 4 * quad + e;
                    if (t < toks) out[(tok0 + t) * w.M + m] = sum[r][tt][e];
                }
    }
}

// y = the shares' sums, added in their order.
__global__ __launch_bounds__(256) void w4_join_kernel(const float *part, int64_t values, int shares, float *y) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < values; i += (int64_t)gridDim.x * 256) {
        float s = part[i];
        for (int k = 1; k < shares; ++k) s += part[k * values + i];
        y[i] = s;
    }
}

template <int FORM>
void launch_pack_form(int groups, dim3 g, hipStream_t st, const void *w, const uint16_t *given, int64_t M,
                      int64_t K, uint8_t *codes, uint16_t *steps) {
#define W4_PACK(GS) \
    hipLaunchKernelGGL((w4_pack_kernel<FORM, GS>), g, dim3(256), 0, st, w, given, M, K, codes, steps)
    if (groups == 1) W4_PACK(1); else if (groups == 2) W4_PACK(2); else W4_PACK(4);
#undef W4_PACK
}

template <bool BF16>
void launch_few(const W4Args &w, const void *x, int64_t N, float *y, hipStream_t st) {
    constexpr int NT = BF16 ? 1 : 2, kLds = 64 * 1024, kRed = kW4Waves * 1024;
    const int nblk = w.K / 128, tiles = (w.M + 15) / 16, block_bytes = 256 * NT * (int)N + 64;
    const int chunk = std::min(nblk, (kLds - kRed) / block_bytes);
    // two workgroups to a compute unit, and the waves of one on as many tiles as leave none idle
    const int64_t groups = 512;
    int wk = 1;
    while (wk < kW4Waves && 2 * wk <= chunk && (int64_t)tiles * wk < groups * kW4Waves) wk *= 2;
    const int slots = kW4Waves / wk;
    const int64_t need = (tiles + slots - 1) / slots;
    const int64_t grid = std::min(need, groups);
    const int iters = (int)((need + grid - 1) / grid);
    const size_t lds = (size_t)chunk * block_bytes + kRed;
#define W4_FEW(GS)                                                                                     \
    hipLaunchKernelGGL((w4_linear_kernel<BF16, 1, GS>), dim3((unsigned)grid), dim3(kW4Threads), lds, st, \
                       w, x, N, y, wk, chunk, iters)
    if (w.groups == 1) W4_FEW(1); else if (w.groups == 2) W4_FEW(2); else W4_FEW(4);
#undef W4_FEW
}

template <bool BF16, int TT, int RT>
void launch_wide(const W4Args &w, const void *x, int64_t N, float *y, float *part, dim3 g, hipStream_t st) {
#define W4_WIDE(GS) \
    hipLaunchKernelGGL((w4_wide_kernel<BF16, TT, GS, RT>), g, dim3(kW4Threads), 0, st, w, x, N, y, part)
    if (w.groups == 1) W4_WIDE(1); else if (w.groups == 2) W4_WIDE(2); else W4_WIDE(4);
#undef W4_WIDE
}
template <bool BF16>
void launch_many(const W4Args &w, const void *x, int64_t N, float *y, float *part, const W4Plan &p,
                 hipStream_t st) {
    const dim3 g((unsigned)p.rows, (unsigned)p.tokens, (unsigned)p.shares);
    if (p.tt == 2) {
        if (p.rt == 2) launch_wide<BF16, 2, 2>(w, x, N, y, part, g, st);
        else launch_wide<BF16, 2, 1>(w, x, N, y, part, g, st);
    } else {
        if (p.rt == 2) launch_wide<BF16, 4, 2>(w, x, N, y, part, g, st);
        else launch_wide<BF16, 4, 1>(w, x, N, y, part, g, st);
    }
    if (p.shares > 1) {
        const int64_t values = N * w.M;
        hipLaunchKernelGGL(w4_join_kernel, dim3((unsigned)std::min<int64_t>((values + 255) / 256, 1 << 16)), dim3(256),
                           0, st, part, values, p.shares, y);
    }
}

}  // namespace

hipError_t launch_w4_pack(const void *w, int form, const uint16_t *given, int64_t M, int64_t K, int groups,
                          uint8_t *codes, uint16_t *steps, hipStream_t st) {
    const int64_t tiles = (M + 15) / 16;
    const dim3 g((unsigned)tiles, (unsigned)std::min<int64_t>((K / 128 + 3) / 4, 64));
    if (form == 0) launch_pack_form<0>(groups, g, st, w, given, M, K, codes, steps);
    else if (form == 1) launch_pack_form<1>(groups, g, st, w, given, M, K, codes, steps);
    else launch_pack_form<2>(groups, g, st, w, given, M, K, codes, steps);
    return hipGetLastError();
}

hipError_t launch_w4_rows(const W4Args &w, const int32_t *ids, int64_t n, void *out, int bf16,
                          hipStream_t st) {
    if (bf16) hipLaunchKernelGGL((w4_rows_kernel<true>), dim3((unsigned)n), dim3(256), 0, st, w, ids, out);
    else hipLaunchKernelGGL((w4_rows_kernel<false>), dim3((unsigned)n), dim3(256), 0, st, w, ids, out);
    return hipGetLastError();
}

hipError_t launch_w4_linear(const W4Args &w, const void *x, int bf16, int64_t N, float *y, float *part,
                            const W4Plan &p, hipStream_t st) {
    if (p.tt == 1) { if (bf16) launch_few<true>(w, x, N, y, st); else launch_few<false>(w, x, N, y, st); }
    else if (bf16) launch_many<true>(w, x, N, y, part, p, st);
    else launch_many<false>(w, x, N, y, part, p, st);
    return hipGetLastError();
}

}  // namespace bitnet
