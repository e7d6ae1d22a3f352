// w4.hip -- matrices of 4-bit weights with a step for each group of channels: the
// quantiser, rows back as floats, and the product with float tokens.
//
//   weight = step * (code - 8),   step fp16, one for each row and GROUP channels
//   y[n][m] = sum_g step_mg * sum_{k in g} x_nk (code_mk - 8)
//
// Layout: tiles of 16 rows, blocks of 128 channels.  codes[tile][block][quad][row][j] is a
// dword with channels 32 j + 8 quad + 0..7 of the block, the first in its low bits: 16
// bytes of a lane (quad, row), 1 KB side by side for a wave, and each dword one operand
// of the 16x16x32 matrix instruction.  steps[tile][block][row][128 / GROUP], or by group
// steps[tile][block][128 / GROUP][row].
//
// The product runs on that instruction for any number of tokens: a code becomes code - 8 in
// fp16 exactly, a token's 128 channels are scaled by a power of two so that the largest is
// in [2^14, 2^15) and carried in one fp16 term (bf16 tokens: exact down to 2^-39 of the
// block's largest) or two (fp32: 22 bits, no finer than 2^-40 of the largest).  A group's sum and
// the sum over groups are fp32.
//
// With the steps by group a lane loads one step of the tile's 16 GS and the groups go round by lane
// swaps: two steps take one and four take three, and no more registers than the other order
// (in graphs, by row and by group: one token times 128000 x 2560 36.4 and 36.8 us, 5 fp32 tokens
// times 50001 x 1024, groups of 32, 11.1 and 11.5, 64 times 8192 x 8192 25.0 and 24.8).
//
// What bounds it.  Few tokens over a large matrix: HBM (one times 128000 x 2560, bf16, 175 MB in
// 35 to 38 us, what a copy reaches; fp32 41; 16 tokens 41 and 49).  A small matrix: the chain of
// launch, tokens, weights and sums (2560 x 2560 5.3 us, 6.1 with fp32).  From 17 tokens on the
// vector operations (unpacking, scales, making the operands) and the LDS, each a third of the
// time with the matrix instructions at a quarter (64 times 8192 x 28672, bf16: 30 GF and
// 127 MB in 54 us and 5 for the join of eight shares; 2048 times 6912 x 2560 142 us, 510 TF).
#include <algorithm>

#include "codes4.h"
#include "layer.h"

namespace bitnet {

namespace {

constexpr int kW4Threads = 512;
constexpr int kW4Waves = kW4Threads / 64;
constexpr float kW4Max = 7.0f * 65504.0f; // 7 steps of the largest fp16

// ---------------------------------------------------------------- quantiser

// A wave takes a tile's block: lane (row, quad), 8 channels of each 32.  FORM 0: fp32, 1:
// bf16 weights; 2: int8 codes -8..7 with steps given as [M][K / GROUP].
template <int FORM, int GS>
__global__ __launch_bounds__(256) void w4_pack_kernel(const void *w, const uint16_t *given, const W4Args to) {
#pragma clang fp contract(off)
    const int lane = threadIdx.x & 63, row = lane & 15, quad = lane >> 4;
    const int64_t M = to.M, K = to.K, nblk = K / 128, m = (int64_t)blockIdx.x * 16 + row;
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
        reinterpret_cast<uint4 *>(to.codes)[out] = make_uint4(word[0], word[1], word[2], word[3]);
        if (quad == 0)
#pragma unroll
            for (int g = 0; g < GS; ++g)
                to.steps[((int64_t)blockIdx.x * nblk + blk) * 16 * GS + (to.by_group ? g * 16 + row : row * GS + g)] = st[g];
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
            const int row = (int)(m & 15), g = w.groups == 4 ? j : w.groups == 2 ? j >> 1 : 0;
            s = (float)__builtin_bit_cast(
                _Float16, w.steps[at * 16 * w.groups + (w.by_group ? g * 16 + row : row * w.groups + g)]);
            if (s != s) s = __uint_as_float(0x7fc00000u);   // bf16_bits would carry other NaNs into the sign
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

// The steps of a tile's block as a lane loads them: its row's, side by side; or by group one of
// the tile's, which the lanes hand each other.
template <int GS>
struct ByGroup {
    uint16_t mine;   // of 16 GS: row n of group `quad` (two groups: quad % 2)
};
template <int GS, bool BY_GROUP>
struct StepWord { using type = ByGroup<GS>; };
template <> struct StepWord<1, false> { using type = uint16_t; };
template <> struct StepWord<2, false> { using type = uint32_t; };
template <> struct StepWord<4, false> { using type = uint2; };
template <typename Word>
__device__ __forceinline__ void load_steps(Word &w, const uint16_t *steps, int64_t block, int lane) {
    w = reinterpret_cast<const Word *>(steps)[block * 16 + (lane & 15)];
}
template <int GS>
__device__ __forceinline__ void load_steps(ByGroup<GS> &w, const uint16_t *steps, int64_t block, int lane) {
    w.mine = steps[block * (16 * GS) + (lane & (16 * GS - 1))];
}
__device__ __forceinline__ float half_of(uint16_t w) { return (float)__builtin_bit_cast(_Float16, w); }
__device__ __forceinline__ void steps_of(uint16_t w, float (&s)[1]) { s[0] = half_of(w); }
__device__ __forceinline__ void steps_of(uint32_t w, float (&s)[2]) {
#pragma unroll
    for (int g = 0; g < 2; ++g) s[g] = (float)as_h2(w)[g];
}
__device__ __forceinline__ void steps_of(const uint2 &w, float (&s)[4]) {
#pragma unroll
    for (int g = 0; g < 4; ++g) s[g] = (float)as_h2(g < 2 ? w.x : w.y)[g & 1];
}
__device__ __forceinline__ void steps_of(const ByGroup<2> &w, float (&s)[2]) {
    partners16(half_of(w.mine), s[0], s[1]);
}
__device__ __forceinline__ void steps_of(const ByGroup<4> &w, float (&s)[4]) {
    float even, odd;
    partners16(half_of(w.mine), even, odd);   // groups 0 0 2 2 and 1 1 3 3
    partners32(even, s[0], s[2]);
    partners32(odd, s[1], s[3]);
}

// The blocks of a turn: many, to be few turns, where a block's operands take little LDS.  (One
// token times 2560 x 2560: 7.5 us with eight blocks in turns of four waves, 5.3 with 32; times
// 128000 x 2560, fp32, a wave to a tile: 43 us with eight, 41 with four.)
constexpr int blocks_of_turn(int slots, int wk, int terms) {
    return slots == 4 ? (wk == 1 ? 4 : 8 * wk)
           : slots == 8 ? (wk == 1 ? 8 : 16)
           : wk == 4    ? 8
           : wk == 2    ? 8 / terms
                        : 4 / terms;
}

// A workgroup has 16 * TT tokens and eight waves over a share of the blocks (blockIdx.z).  WK of
// the waves share a tile's blocks, so that few rows have many waves; or a wave has RT tiles,
// which halves what it reads of the operands in LDS (w4_plan.h chooses).
// The tokens' operands are made CB blocks at a time in one half of the LDS while the matrix
// instructions read the other half: the values for it are on their way meanwhile, and so is
// each block of weights a turn ahead of its use.  Token t of the 16 bytes (j, quad) = p lies
// in slot (t + 4 p) mod SLOTS, so that the lanes that write eight channels each of a few tokens
// spread over all banks; up to four tokens take four slots, up to eight eight.
template <bool BF16, int TT, int GS, bool BY_GROUP, int RT, int WK, int SLOTS>
__global__ __launch_bounds__(kW4Threads, 2) void w4_linear_kernel(const W4Args w, const void *x, int64_t N,
                                                                  float *y, float *part) {
    constexpr int NT = BF16 ? 1 : 2, TOK = 16 * TT;
    constexpr int CB = blocks_of_turn(SLOTS, WK, NT), OWN = CB / WK;
    constexpr int kPieces = (CB * SLOTS * 16 + kW4Threads - 1) / kW4Threads;   // of 8 channels, for a thread
    __shared__ h8 xs[2][CB * 16 * NT][SLOTS];
    __shared__ __align__(16) float sc[2][CB][TOK];
    const int lane = threadIdx.x & 63, n = lane & 15, quad = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t tok0 = (int64_t)blockIdx.y * TOK;
    const int toks = (int)min(N - tok0, (int64_t)TOK);
    const int nblk = w.K / 128, tiles = (w.M + 15) / 16;
    const int begin = (int)((int64_t)nblk * blockIdx.z / gridDim.z), end = (int)((int64_t)nblk * (blockIdx.z + 1) / gridDim.z);
    const int turn = wave % WK;   // of the waves of a tile: its blocks are turn, turn + WK, ...
    const int tile0 = ((int)blockIdx.x * (kW4Waves / WK) + wave / WK) * RT;
    using Word = typename StepWord<GS, BY_GROUP>::type;
    uint4 raw[OWN][RT];
    Word st[OWN][RT];
    auto load_weights = [&](int i, int b0) {
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const int64_t at = (int64_t)min(tile0 + r, tiles - 1) * nblk + min(b0 + i * WK + turn, end - 1);
            raw[i][r] = reinterpret_cast<const uint4 *>(w.codes)[at * 64 + lane];
            load_steps(st[i][r], w.steps, at, lane);
        }
    };
    uint4 v[kPieces][NT];   // eight channels as they are
    const int p = threadIdx.x & 15, u0 = threadIdx.x >> 4;   // piece i: unit u0 + 32 i, a token's block
    auto load_tokens = [&](int b0) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int u = u0 + 32 * i, c = u / SLOTS, t = min(u % SLOTS, toks - 1);
            const int64_t at = (tok0 + t) * w.K + (int64_t)min(b0 + c, end - 1) * 128 + 8 * p;
#pragma unroll
            for (int k = 0; k < NT; ++k) v[i][k] = reinterpret_cast<const uint4 *>(x)[at / (8 / NT) + k];
        }
    };
    auto put_tokens = [&](int half) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int u = u0 + 32 * i, c = u / SLOTS, t = u % SLOTS;
            if (c >= CB || (TT == 1 && t >= toks)) continue;   // the same for the 16 lanes
            h8 h[NT];
            float f[8];
            load8<BF16>(v[i], 0, f);
            const float down = halves_of<NT>(f, h);
#pragma unroll
            for (int k = 0; k < NT; ++k) xs[half][(c * 4 + (p >> 2)) * NT * 4 + k * 4 + (p & 3)][(t + 4 * p) % SLOTS] = h[k];
            if (p == 0) sc[half][c][t] = down;
        }
    };
    load_tokens(begin);
#pragma unroll
    for (int i = 0; i < OWN; ++i) load_weights(i, begin);
    put_tokens(0);
    __syncthreads();
    const uint32_t one = ones_1024();
    int tok[TT];   // the operand's token of this lane: the last one again behind it
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) tok[tt] = (TT == 1 ? min(n, toks - 1) : 16 * tt + n) + 4 * quad;
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
        for (int i = 0; i < OWN; ++i) {
            const int c = i * WK + turn;
            if (b0 + c >= end) continue;
            f4 block[RT][TT];
            float step[RT][GS];
#pragma unroll
            for (int r = 0; r < RT; ++r) steps_of(st[i][r], step[r]);
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
                        const uint32_t word = j == 0 ? raw[i][r].x : j == 1 ? raw[i][r].y : j == 2 ? raw[i][r].z : raw[i][r].w;
                        h2 q[4];
                        codes8<false>(word, one, q);
                        wq[r] = join(q[0], q[1], q[2], q[3]);
                    }
#pragma unroll
                    for (int tt = 0; tt < TT; ++tt)
#pragma unroll
                        for (int k = 0; k < NT; ++k) {
                            const h8 a = xs[half][(c * 4 + j) * NT * 4 + k * 4 + quad][(tok[tt] + 16 * j) % SLOTS];
#pragma unroll
                            for (int r = 0; r < RT; ++r) acc[r][tt] = mfma(a, wq[r], acc[r][tt]);
                        }
                }
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int tt = 0; tt < TT; ++tt)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            block[r][tt][e] = g == 0 ? acc[r][tt][e] * step[r][g] : fmaf(acc[r][tt][e], step[r][g], block[r][tt][e]);
            }
#pragma unroll
            for (int tt = 0; tt < TT; ++tt) {
                const f4 s = *reinterpret_cast<const f4 *>(&sc[half][c][16 * tt + 4 * quad]);
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sum[r][tt][e] = fmaf(block[r][tt][e], s[e], sum[r][tt][e]);
            }
            load_weights(i, b0 + CB);
        }
        if (more) put_tokens(half ^ 1);
        __syncthreads();
    }
    if constexpr (WK > 1) {   // the waves of a tile, in their order
        f4 *const red = reinterpret_cast<f4 *>(xs);
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int tt = 0; tt < TT; ++tt) red[((wave * RT + r) * TT + tt) * 64 + lane] = sum[r][tt];
        __syncthreads();
        if (turn != 0) return;
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int tt = 0; tt < TT; ++tt)
#pragma unroll
                for (int k = 1; k < WK; ++k) sum[r][tt] += red[(((wave + k) * RT + r) * TT + tt) * 64 + lane];
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
void launch_pack_form(dim3 g, hipStream_t st, const void *w, const uint16_t *given, const W4Args &to) {
#define W4_PACK(GS) hipLaunchKernelGGL((w4_pack_kernel<FORM, GS>), g, dim3(256), 0, st, w, given, to)
    if (to.groups == 1) W4_PACK(1); else if (to.groups == 2) W4_PACK(2); else W4_PACK(4);
#undef W4_PACK
}

template <bool BF16, int TT, int RT, int WK, int SLOTS = 16 * TT>
void launch_linear_t(const W4Args &w, const void *x, int64_t N, float *y, float *part, const W4Plan &p,
                     hipStream_t st) {
    const dim3 g((unsigned)p.rows, (unsigned)p.tokens, (unsigned)p.shares), t(kW4Threads);
#define W4_LINEAR(GS, BY_GROUP) \
    hipLaunchKernelGGL((w4_linear_kernel<BF16, TT, GS, BY_GROUP, RT, WK, SLOTS>), g, t, 0, st, w, x, N, y, part)
    if (w.groups == 1) W4_LINEAR(1, false);   // both orders are the same
    else if (w.by_group) { if (w.groups == 2) W4_LINEAR(2, true); else W4_LINEAR(4, true); }
    else if (w.groups == 2) W4_LINEAR(2, false);
    else W4_LINEAR(4, false);
#undef W4_LINEAR
}
template <bool BF16>
void launch_linear(const W4Args &w, const void *x, int64_t N, float *y, float *part, const W4Plan &p,
                   hipStream_t st) {
    if (N <= 4) {
        if (p.wk == 4) launch_linear_t<BF16, 1, 1, 4, 4>(w, x, N, y, part, p, st);
        else if (p.wk == 2) launch_linear_t<BF16, 1, 1, 2, 4>(w, x, N, y, part, p, st);
        else launch_linear_t<BF16, 1, 1, 1, 4>(w, x, N, y, part, p, st);
    } else if (N <= 8) {
        if (p.wk == 4) launch_linear_t<BF16, 1, 1, 4, 8>(w, x, N, y, part, p, st);
        else if (p.wk == 2) launch_linear_t<BF16, 1, 1, 2, 8>(w, x, N, y, part, p, st);
        else launch_linear_t<BF16, 1, 1, 1, 8>(w, x, N, y, part, p, st);
    } else if (p.tt == 1 && p.wk == 4) launch_linear_t<BF16, 1, 1, 4>(w, x, N, y, part, p, st);
    else if (p.tt == 1 && p.wk == 2) launch_linear_t<BF16, 1, 1, 2>(w, x, N, y, part, p, st);
    else if (p.tt == 1) launch_linear_t<BF16, 1, 1, 1>(w, x, N, y, part, p, st);
    else if (p.tt == 2 && p.rt == 2) launch_linear_t<BF16, 2, 2, 1>(w, x, N, y, part, p, st);
    else if (p.tt == 2) launch_linear_t<BF16, 2, 1, 1>(w, x, N, y, part, p, st);
    else if (p.rt == 2) launch_linear_t<BF16, 4, 2, 1>(w, x, N, y, part, p, st);
    else launch_linear_t<BF16, 4, 1, 1>(w, x, N, y, part, p, st);
}

}  // namespace

hipError_t launch_w4_pack(const void *w, int form, const uint16_t *given, const W4Args &to, hipStream_t st) {
    const int tiles = (to.M + 15) / 16;
    const dim3 g((unsigned)tiles, (unsigned)std::min((to.K / 128 + 3) / 4, 64));
    if (form == 0) launch_pack_form<0>(g, st, w, given, to);
    else if (form == 1) launch_pack_form<1>(g, st, w, given, to);
    else launch_pack_form<2>(g, st, w, given, to);
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
    if (bf16) launch_linear<true>(w, x, N, y, part, p, st);
    else launch_linear<false>(w, x, N, y, part, p, st);
    if (p.shares > 1) {
        const int64_t values = N * w.M;
        hipLaunchKernelGGL(w4_join_kernel, dim3((unsigned)std::min<int64_t>((values + 255) / 256, 1 << 16)), dim3(256),
                           0, st, part, values, p.shares, y);
    }
    return hipGetLastError();
}

}  // namespace bitnet
