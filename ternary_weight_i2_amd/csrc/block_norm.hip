// block_norm.hip -- the boundary between two blocks of a layer: the norm after
// the block, its gate and residual scale, the residual stream, the norm before
// the next block and the int8 tokens that its matmuls take.
//
// Pages: [P4] "bitnet.rs", "Forward Pass" (norm, residual add, the sub-norm in
// front of the output projection); [P1] "BitNet 딥다이브" §4-5 (per-token
// absmax int8 activations).
//
// Per token, every step one fp32 rounding:
//   t = b;  post: t = (t * c1) * g1;  gate: t = t * gate;  t = t * scale
//   h = round_to_stream(res + t)      (or t itself without a residual)
//   v = (h * c2) * g2                 s = 127 / max(max|v|, 1e-5)
//   xq = round(v * s)                 x_sum = sum xq
// c = fp32(1 / sqrt(mean + eps)), the mean of squares in binary64 (a square of
// an fp32 value is exact there).
//
// One workgroup per token keeps the token in registers between the steps, so
// every input is read once and every output written once; what bounds it is
// HBM for long prompts (4096 tokens of 2560, fp32 into a bf16 stream, a gate per
// token: 136 MB in 28 us, 4.8 TB/s, what a large copy reaches) and the chain of
// loads and workgroup reductions (two sums, one maximum, one sum of codes) for
// single tokens (3.4 us at 2560, of which the reductions are 1.0; 64 tokens of 8192,
// norms on both sides, which leave three of four compute units idle: 6.7 us, of which
// the reductions are 1.5).
// The workgroup's width depends on F alone, so a token's result does not depend on
// N; workgroups of half or twice the width took as long or up to 1.7 times it.
#include <algorithm>

#include "layer.h"

namespace bitnet {

namespace {

constexpr int kNormMaxThreads = 1024;
constexpr int kNormMaxWaves = kNormMaxThreads / 64;

struct NormShared {
    double sum[2][kNormMaxWaves];
    float amax[kNormMaxWaves];
    int codes[kNormMaxWaves];
};

// Stores eight values; bf16 rounds to nearest even and leaves the stored
// values in x.
template <bool BF16>
__device__ __forceinline__ void store8(void *p, int64_t i, float (&x)[8]) {
    if constexpr (BF16) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t a = bf16_bits(x[2 * e]), b = bf16_bits(x[2 * e + 1]);
            w[e] = a | b << 16;
            x[2 * e] = __uint_as_float(a << 16);
            x[2 * e + 1] = __uint_as_float(b << 16);
        }
        if (p)
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + i) =
                make_uint4(w[0], w[1], w[2], w[3]);
    } else if (p) {
        float4 *f = reinterpret_cast<float4 *>(static_cast<float *>(p) + i);
        f[0] = make_float4(x[0], x[1], x[2], x[3]);
        f[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
}

// fp32(1 / sqrt(ss / F + eps)) of the workgroup's sum of squares.  The waves'
// sums meet in LDS and every thread adds them in the same order.
__device__ __forceinline__ float block_factor(double ss, double (&part)[kNormMaxWaves], int F,
                                              float eps) {
    ss = wave_sum_f64(ss);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = ss;
    __syncthreads();
    double t = part[0];
    for (int w = 1; w < (int)(blockDim.x >> 6); ++w) t += part[w];
    return (float)(1.0 / sqrt(t / (double)F + (double)eps));
}

template <int R, bool BB, bool SB>
__global__ __launch_bounds__(R == 4 ? kNormMaxThreads : 512) void block_norm_kernel(
    const BlockNormArgs a) {
#pragma clang fp contract(off)
    __shared__ NormShared sh;
    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
    const int pieces = a.F >> 3;
    const int64_t row = (int64_t)blockIdx.x * a.F;
    // Everything the token needs is requested before the first sum is waited for
    // (rows of over 8192 channels: what the registers of a wider workgroup hold).
    constexpr bool kAhead = R < 4;
    float t[R][8], res[R][8], pg[kAhead ? R : 1][8], gt[kAhead ? R : 1][8], gm[kAhead ? R : 1][8];
    auto load_gain = [&](const float *p, int64_t i, float (&x)[8]) {
        if (p) {
            load8<false>(p, i, x);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = 1.0f;
        }
    };
    const float *gate = a.gate ? a.gate + blockIdx.x * a.gate_stride : nullptr;
    double ss = 0.0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int p = tid + r * blockDim.x, q = min(p, pieces - 1);
        load8<BB>(a.b, row + 8 * q, t[r]);
        if (a.res) load8<SB>(a.res, row + 8 * q, res[r]);
        if constexpr (kAhead) {
            load_gain(a.post_gamma, 8 * q, pg[r]);
            load_gain(gate, 8 * q, gt[r]);
            load_gain(a.gamma, 8 * q, gm[r]);
        }
    }
    // ---- the block's output, its norm, gate and scale
    float c1 = 1.0f;
    if (a.post) {
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (tid + r * blockDim.x < pieces)
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = fma((double)t[r][e], (double)t[r][e], ss);
        c1 = block_factor(ss, sh.sum[0], a.F, a.eps);
    }
    ss = 0.0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int p = tid + r * blockDim.x;
        if (p < pieces) {
            float(&g1)[8] = pg[kAhead ? r : 0], (&g2)[8] = gt[kAhead ? r : 0];
            if constexpr (!kAhead) {
                load_gain(a.post_gamma, 8 * p, g1);
                load_gain(gate, 8 * p, g2);
            }
            // a factor of 1 changes nothing, so what is absent needs no branch
#pragma unroll
            for (int e = 0; e < 8; ++e) t[r][e] = (((t[r][e] * c1) * g1[e]) * g2[e]) * a.scale;
            // ---- the residual stream, as it is stored
            if (a.res) {
#pragma unroll
                for (int e = 0; e < 8; ++e) t[r][e] = res[r][e] + t[r][e];
                store8<SB>(a.h, row + 8 * p, t[r]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fma((double)t[r][e], (double)t[r][e], ss);
        }
    }
    // ---- the norm before the next block
    const float c2 = block_factor(ss, sh.sum[1], a.F, a.eps);
    float amax = 0.0f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int p = tid + r * blockDim.x;
        if (p < pieces) {
            float(&g)[8] = gm[kAhead ? r : 0];
            if constexpr (!kAhead) load_gain(a.gamma, 8 * p, g);
#pragma unroll
            for (int e = 0; e < 8; ++e) t[r][e] = (t[r][e] * c2) * g[e];
#pragma unroll
            for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(t[r][e]));
            if (a.v) {
                float o[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = t[r][e];
                store8<SB>(a.v, row + 8 * p, o);
            }
        }
    }
    if (!a.xq) return;   // uniform over the workgroup
    amax = wave_max_f32(amax);
    if (lane == 0) sh.amax[wv] = amax;
    __syncthreads();
    amax = sh.amax[0];
    for (int w = 1; w < (int)(blockDim.x >> 6); ++w) amax = fmaxf(amax, sh.amax[w]);
    const float s = quant_scale(amax);
    int sum = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int p = tid + r * blockDim.x;
        if (p < pieces) {
            uint32_t c[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float *x = &t[r][4 * i];
                c[i] = pack_low_bytes(quant_bits(x[0], s), quant_bits(x[1], s),
                                      quant_bits(x[2], s), quant_bits(x[3], s));
                sum = sum_codes4(c[i], sum);
            }
            *reinterpret_cast<uint2 *>(a.xq + row + 8 * p) = make_uint2(c[0], c[1]);
        }
    }
    sum = wave_sum_i32(sum);
    if (lane == 0) sh.codes[wv] = sum;
    __syncthreads();
    if (tid == 0) {
        int total = 0;
        for (int w = 0; w < (int)(blockDim.x >> 6); ++w) total += sh.codes[w];
        a.xs[blockIdx.x] = s;
        a.xsum[blockIdx.x] = total;
    }
}

template <int R>
void launch_r(const BlockNormArgs &a, int64_t N, int threads, int b_bf16, int s_bf16,
              hipStream_t st) {
    const dim3 g((unsigned)N), t((unsigned)threads);
    if (b_bf16 && s_bf16) hipLaunchKernelGGL((block_norm_kernel<R, true, true>), g, t, 0, st, a);
    else if (b_bf16) hipLaunchKernelGGL((block_norm_kernel<R, true, false>), g, t, 0, st, a);
    else if (s_bf16) hipLaunchKernelGGL((block_norm_kernel<R, false, true>), g, t, 0, st, a);
    else hipLaunchKernelGGL((block_norm_kernel<R, false, false>), g, t, 0, st, a);
}

}  // namespace

hipError_t launch_block_norm(const BlockNormArgs &a, int64_t N, int b_bf16, int s_bf16,
                             hipStream_t st) {
    // eight channels per thread up to 4096, 16 up to 8192, then up to 32
    const int pieces = a.F >> 3;
    const int r = pieces <= 512 ? 1 : pieces <= 1024 ? 2 : 4;
    const int threads = ((pieces + r - 1) / r + 63) / 64 * 64;
    // a launch has fewer than 2^32 threads: 2^21 tokens at a time
    constexpr int64_t kTokens = 1 << 21;
    for (int64_t n0 = 0; n0 < N; n0 += kTokens) {
        const int64_t n = std::min(N - n0, kTokens), at = n0 * a.F;
        auto rows = [&](auto *p, int bytes) {
            using T = decltype(p);
            return p ? (T)((uintptr_t)p + (uintptr_t)(at * bytes)) : p;
        };
        BlockNormArgs c = a;
        const int sb = s_bf16 ? 2 : 4;
        c.b = rows(a.b, b_bf16 ? 2 : 4);
        c.res = rows(a.res, sb);
        c.h = rows(a.h, sb);
        c.v = rows(a.v, sb);
        c.xq = rows(a.xq, 1);
        if (a.gate) c.gate = a.gate + n0 * a.gate_stride;
        if (a.xq) {
            c.xs = a.xs + n0;
            c.xsum = a.xsum + n0;
        }
        if (r == 1) launch_r<1>(c, n, threads, b_bf16, s_bf16, st);
        else if (r == 2) launch_r<2>(c, n, threads, b_bf16, s_bf16, st);
        else launch_r<4>(c, n, threads, b_bf16, s_bf16, st);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace bitnet
