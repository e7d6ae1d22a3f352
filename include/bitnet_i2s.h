/*
 * bitnet_i2s.h -- C ABI of libbitnet_i2s.so, the MI355X (gfx950) BitNet b1.58
 * W2A8 matmul: ternary weights packed as I2_S, per-token absmax int8
 * activations, exact int32 dots and fp32 scaled outputs.
 *
 * Sources (web pages, cited by key and section):
 *   [P1] "BitNet 딥다이브 -- 작은 숫자를 빠른 연산으로 바꾸는 추론 엔진"
 *        (fiv.co.kr/repos/BitNet-deep-dive.html)
 *   [P2] "[분석/검증-3] BitNet.cpp ARM 커널 재작성 : 스칼라 폴백구현을 통한
 *        최종 검증" (uno-kim.tistory.com/459)
 *   [P3] "[기술 분석 보고서] ARM64 모바일 환경에서의 1.58-bit 양자화 모델 추론
 *        붕괴 원인 분석 및 C++ 커널 역공학을 통한 해결" (uno-kim.tistory.com/461)
 *   [P4] "bitnet.rs -- BitNet b1.58 Inference Engine in Rust",
 *        section "Mathematical Foundation"
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Notation: M = output rows (weight rows), K = reduction length, N = tokens.
 *    K must be a positive multiple of 128 (one I2_S block, [P1 §4-2]) and at
 *    most BITNET_MAX_K.
 *  - All pointers except `stream` are DEVICE pointers to caller-owned memory,
 *    row-major and densely packed.  The library never allocates, frees or
 *    retains caller memory and keeps no handles; it is reentrant.
 *  - `stream` is a hipStream_t passed as void* (NULL = the null stream).  Every
 *    call only enqueues work and returns without synchronising, except
 *    bitnet_pack_i2s (see there).
 *  - Arguments are validated on the host before anything is enqueued.  On any
 *    non-zero return nothing has been launched and no output written (except
 *    BITNET_E_VALUE / BITNET_E_HIP after a launch, documented per call).
 *    bitnet_last_error() then describes the failure.
 *  - M == 0 or N == 0 is a valid no-op returning BITNET_OK.
 *  - Results are deterministic: integer sums are exact and order-free, so
 *    repeated calls produce bit-identical int32 and fp32 outputs.
 */
#ifndef BITNET_I2S_H
#define BITNET_I2S_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define BITNET_ABI_VERSION 2
#define BITNET_MAX_K 32768          /* largest supported reduction length   */
#define BITNET_GEMV_MAX_N 64        /* largest token count of the decode call */
#define BITNET_GEMM_MAX_N (1 << 21) /* largest token count of the prefill call */
#define BITNET_MAX_GROUP 8          /* matrices per bitnet_linear_i2s call     */
#define BITNET_LINEAR_FUSED_MAX_N 2 /* bitnet_linear_i2s: one fused launch up to this N */
#define BITNET_LUT_MAX_K 8192       /* largest K of the table-lookup decode call */
#define BITNET_KV4_PAGE 64          /* tokens of a page of the 4-bit cache     */
#define BITNET_KV4_GROUP 64         /* channels that share a step and a middle */
#define BITNET_KV4_MAX_HEADS 1024   /* query heads, and kv heads, of a call    */
#define BITNET_KV4_MAX_SEQS (1 << 20)  /* sequences of a call                  */
#define BITNET_KV4_MAX_PAGES (1 << 24) /* pages of a sequence (2^30 tokens)    */
#define BITNET_W4_MAX_ROWS (1 << 24) /* rows of a matrix of 4-bit weights      */
#define BITNET_W4_BY_GROUP 0x1000   /* bitnet_w4_matrix.group: order of the steps */
#define BITNET_ROTARY_MAX_DIM 1024  /* channels of a head that positions turn   */

typedef enum {
    BITNET_OK = 0,
    BITNET_E_NULL = 1,   /* a required pointer is NULL                        */
    BITNET_E_SHAPE = 2,  /* negative size, K % 128 != 0, K or N out of range  */
    BITNET_E_ALIGN = 3,  /* a pointer lacks the alignment stated below        */
    BITNET_E_DTYPE = 4,  /* unknown activation dtype                          */
    BITNET_E_VALUE = 5,  /* pack saw a weight outside {-1, 0, +1}             */
    BITNET_E_HIP = 6     /* HIP launch/runtime error (text in last_error)     */
} bitnet_status;

typedef enum { BITNET_F32 = 0, BITNET_BF16 = 1 } bitnet_dtype;

/*
 * bitnet_pack_i2s -- ternary int8 weights -> I2_S bytes  [P1 §1-1, §4-2]
 *
 *   w       [M][K] int8, every entry in {-1, 0, +1}; 4-byte aligned.
 *   packed  [M][K/4] uint8 output; 16-byte aligned.  Weight (m, k) is stored
 *           as code w+1 (-1 -> 0b00, 0 -> 0b01, +1 -> 0b10 [P1 §1-1]) in byte
 *           m*K/4 + 32*(k/128) + (k%128)%32, at bit 6 - 2*((k%128)/32):
 *           byte j of a 128-weight block carries elements j, j+32, j+64, j+96,
 *           the first in bits 7-6 [P1 §4-2].  Code 0b11 is never written.
 *
 * Packing is a one-time, offline step, so this call synchronises `stream` to
 * read back a device-side count of non-ternary inputs and returns
 * BITNET_E_VALUE if there were any; the contents of `packed` are then
 * unspecified.  Calls on one device serialise on that count internally.
 */
int bitnet_pack_i2s(const int8_t *w, int64_t M, int64_t K, uint8_t *packed,
                    void *stream);

/*
 * bitnet_quant_act_i8 -- per-token absmax int8 quantisation  [P1 §4-5; P4]
 *
 *   x        [N][K] activations, fp32 (dtype BITNET_F32) or bf16 (BITNET_BF16);
 *            16-byte aligned.  bf16 is widened exactly to fp32 first.
 *   xq       [N][K] int8 output, 16-byte aligned.
 *   x_scale  [N] fp32 output: s_n = 127 / max(max_k |x[n][k]|, 1e-5), the
 *            correctly rounded fp32 quotient (a multiplier, not 1/s).
 *   x_sum    [N] int32 output: sum_k xq[n][k] (needed by the raw-code dot).
 *
 * xq[n][k] = clamp(round_half_even(x[n][k] * s_n), -128, 127) with x*s a
 * single fp32 product (only -127..127 is reachable).  Non-finite inputs give
 * unspecified results.
 */
int bitnet_quant_act_i8(const void *x, int dtype, int64_t N, int64_t K,
                        int8_t *xq, float *x_scale, int32_t *x_sum,
                        void *stream);

/*
 * bitnet_gemv_i2s_i8 -- decode matmul, 1 <= N <= BITNET_GEMV_MAX_N tokens
 * bitnet_gemm_i2s_i8 -- prefill matmul, 0 <= N <= BITNET_GEMM_MAX_N (int8 MFMA)
 *
 *   packed   [M][K/4] I2_S weights (as written by bitnet_pack_i2s), 16-byte
 *            aligned.  A slot holding code 0b11 gives unspecified results.
 *   w_scale  per-tensor weight scale alpha (AbsMean, weight = code-1 times
 *            alpha [P1 §6-2; P4]).
 *   xq, x_scale, x_sum  as produced by bitnet_quant_act_i8 for N tokens;
 *            xq 16-byte aligned.
 *   dot      [N][M] int32 output or NULL:
 *              dot[n][m] = sum_k (code(m,k) - 1) * xq[n][k]
 *            computed as the raw-code sum minus x_sum[n], the exact offset
 *            correction of [P2 §3; P3 §3.2] (never the zero-mean shortcut).
 *   y        [N][M] fp32 output or NULL: y[n][m] = dot[n][m] * w_scale /
 *            x_scale[n], the caller-side scaling of [P2 §3] (relative error
 *            below 1e-6; exactly 0 where dot is 0).
 *   At least one of dot / y must be non-NULL.
 *
 * gemv returns BITNET_E_SHAPE for N > BITNET_GEMV_MAX_N, gemm for
 * N > BITNET_GEMM_MAX_N; both for M > 2^31-1.
 */
int bitnet_gemv_i2s_i8(const uint8_t *packed, float w_scale, int64_t M,
                       int64_t K, const int8_t *xq, const float *x_scale,
                       const int32_t *x_sum, int64_t N, int32_t *dot, float *y,
                       void *stream);

int bitnet_gemm_i2s_i8(const uint8_t *packed, float w_scale, int64_t M,
                       int64_t K, const int8_t *xq, const float *x_scale,
                       const int32_t *x_sum, int64_t N, int32_t *dot, float *y,
                       void *stream);

/*
 * bitnet_gemv_i2s_lut -- the decode matmul of bitnet_gemv_i2s_i8 computed by
 * table lookup instead of unpacking the codes [P1 §4-3, §4-4 (the LUT route:
 * tables are built from the activations alone, then, after a barrier, the
 * weights index them); P1 §11-2 (T-MAC)].  For each token the call tabulates,
 * for every pair of 2-bit fields sharing a nibble of an I2_S byte, the 16
 * raw-code sums c_hi * x_first + c_lo * x_second, then sums one table entry
 * per nibble of each row; D = that sum minus x_sum[n].
 *
 * Arguments, layouts, outputs and errors are those of bitnet_gemv_i2s_i8
 * (identical dot and y, bit for bit), plus BITNET_E_SHAPE for
 * K > BITNET_LUT_MAX_K (the tables of a token live in 16*K bytes of LDS).
 * Weights are read once per token (no reuse across tokens): meant for N = 1.
 */
int bitnet_gemv_i2s_lut(const uint8_t *packed, float w_scale, int64_t M,
                        int64_t K, const int8_t *xq, const float *x_scale,
                        const int32_t *x_sum, int64_t N, int32_t *dot, float *y,
                        void *stream);

/*
 * bitnet_linear_i2s -- fused decode linear: quantise tokens and multiply them
 * by up to BITNET_MAX_GROUP I2_S matrices that share them, in one launch.
 * [P1 §4-5 (per-token scale), §4-3 (a weight block reused for several
 * activation columns); P2 §3; P3 §3.2]
 *
 *   x        [N][K] fp32 or bf16 tokens (as bitnet_quant_act_i8), 16-byte aligned.
 *   mats     host array of n_mats descriptors, read during the call only:
 *              packed [M][K/4] I2_S (16-byte aligned), M, w_scale, and the
 *              outputs dot [N][M] int32 / y [N][M] fp32 (either may be NULL,
 *              not both, unless M == 0).
 *   xq, x_scale, x_sum   optional outputs (may be NULL when
 *              N <= BITNET_LINEAR_FUSED_MAX_N): the
 *              quantised tokens exactly as bitnet_quant_act_i8 writes them.
 *              Required for larger N (they then carry the tokens between the
 *              quantiser and the MFMA kernels).
 *
 * N <= BITNET_LINEAR_FUSED_MAX_N: one launch quantises and multiplies (the
 * vector-ALU GEMV; at more tokens it is ALU-bound and slower than the two
 * launches below).  Up to BITNET_GEMV_MAX_N:
 * quantiser, then one batched-decode MFMA launch for all matrices.  Larger N
 * (prefill): quantiser, then one grouped MFMA GEMM launch for all matrices.
 * Every output equals what bitnet_quant_act_i8 followed by
 * bitnet_gemv_i2s_i8 (N <= BITNET_GEMV_MAX_N) or bitnet_gemm_i2s_i8 on each
 * matrix produces, bit for bit.
 * 0 <= N <= BITNET_GEMM_MAX_N; 1 <= n_mats <= BITNET_MAX_GROUP.
 */
typedef struct {
    const uint8_t *packed;
    int64_t M;
    float w_scale;
    int32_t *dot;
    float *y;
} bitnet_i2s_matrix;

int bitnet_linear_i2s(const void *x, int dtype, int64_t N, int64_t K,
                      const bitnet_i2s_matrix *mats, int n_mats, int8_t *xq,
                      float *x_scale, int32_t *x_sum, void *stream);

/*
 * bitnet_ffn_act_quant_i8 -- the squared-ReLU gated FFN activation that feeds
 * the down projection, quantised for it.  [P4 "Forward Pass":
 * inner = ffn_sub_norm(sqrelu(gate(x)) * up(x)), out = down(inner); P1 §4-5]
 *
 *   g, u     device [N][F] fp32: the gate and up projections' y outputs
 *            (16-byte aligned); F a multiple of 128, F <= BITNET_MAX_K.
 *   gamma    device [F] fp32 gain of the sub-norm (16-byte aligned), or NULL for 1.
 *   eps      the sub-norm's epsilon (positive, finite; else BITNET_E_VALUE).
 *   xq, x_scale, x_sum   outputs as bitnet_quant_act_i8 writes them, ready
 *            for bitnet_gemv_i2s_i8 / bitnet_gemm_i2s_i8 with the down weights.
 *
 * Per token: h = (relu(g)^2) * u in fp32; ss = the sum of the F squares h^2
 * (each exact in binary64) computed exactly and rounded once to binary64,
 * to nearest-even -- no summation order enters; c = fp32(1 / sqrt(ss / F +
 * eps)); v = (h * c) * gamma in fp32; then per-token absmax int8 quantisation
 * of v.  0 <= N < 2^31; N == 0 is a no-op.
 */
int bitnet_ffn_act_quant_i8(const float *g, const float *u, const float *gamma, float eps,
                            int64_t N, int64_t F, int8_t *xq, float *x_scale,
                            int32_t *x_sum, void *stream);

/*
 * bitnet_gemv_i2s_i8_group -- decode matmul (N <= BITNET_GEMV_MAX_N tokens,
 * already quantised) of several I2_S matrices that share the tokens: one
 * launch for all of them: the vector-ALU GEMV when N <= 2, else the
 * batched-decode MFMA kernel.  [P1 §2-1, §4-3; P2 §3; P3 §3.2]
 *
 *   mats, xq, x_scale, x_sum   as bitnet_gemm_i2s_i8_group.
 *
 * Outputs equal bitnet_gemv_i2s_i8 on each matrix, bit for bit.
 * 0 <= N <= BITNET_GEMV_MAX_N; N == 0 or all M == 0 is a no-op.
 */
int bitnet_gemv_i2s_i8_group(const bitnet_i2s_matrix *mats, int n_mats, int64_t K,
                             const int8_t *xq, const float *x_scale,
                             const int32_t *x_sum, int64_t N, void *stream);

/*
 * bitnet_gemm_i2s_i8_group -- prefill matmul of several I2_S matrices that
 * share one block of quantised tokens, in one MFMA launch (e.g. q/k/v, or
 * gate/up, of a layer).  [P1 §4-5 (a separate prefill path), §4-3 (one
 * token block reused by every weight row); P2 §3; P3 §3.2]
 *
 *   mats     host array of n_mats descriptors (1 <= n_mats <=
 *            BITNET_MAX_GROUP), read during the call only: packed [M][K/4]
 *            I2_S (16-byte aligned), M, w_scale, outputs dot [N][M] int32 /
 *            y [N][M] fp32 (either may be NULL, not both, unless M == 0).
 *   xq, x_scale, x_sum   the tokens as bitnet_quant_act_i8 writes them
 *            (xq 16-byte aligned).
 *
 * Outputs equal bitnet_gemm_i2s_i8 on each matrix, bit for bit.
 * 0 <= N <= BITNET_GEMM_MAX_N; N == 0 or all M == 0 is a no-op.
 */
int bitnet_gemm_i2s_i8_group(const bitnet_i2s_matrix *mats, int n_mats, int64_t K,
                             const int8_t *xq, const float *x_scale,
                             const int32_t *x_sum, int64_t N, void *stream);

/*
 * bitnet_absmean_i2s -- one-time conversion of full-precision weights to I2_S
 * with the AbsMean ternariser.  [P1 §6-2; P4 "Ternary Weight Quantisation
 * (AbsMean)"; layout P1 §1-1, §4-2]
 *
 *   w       device [M][K] fp32 or bf16 (dtype BITNET_F32 / BITNET_BF16),
 *           16-byte aligned; M >= 1.
 *   packed  device [M][K/4] I2_S output, 16-byte aligned.
 *   alpha   HOST pointer; receives the per-tensor scale
 *           alpha = max(mean |w| over all M*K weights, 1e-5): the sum of |w|
 *           computed exactly and rounded once to binary64 (so it depends on
 *           no summation order), divided by M*K in binary64, rounded to fp32.
 *           Use it as w_scale of the matmul calls.
 *
 * Each weight becomes q = clip(round-half-even(w / alpha), -1, 1), w / alpha
 * one fp32 division, stored as code q + 1.  Synchronises `stream`
 * (the scale is returned on the host); calls are serialised inside the
 * library.  Non-finite weights -> BITNET_E_VALUE (packed then unspecified);
 * M * K above 2^40 -> BITNET_E_SHAPE.
 */
int bitnet_absmean_i2s(const void *w, int dtype, int64_t M, int64_t K,
                       uint8_t *packed, float *alpha, void *stream);

/*
 * bitnet_pack_i2s_f32 -- pack float weights that are already ternary in value
 * (e.g. q * scale) by sign: |v| < 1e-6 (compared in binary64) -> code 1,
 * v > 0 -> code 2, v < 0 -> code 0.  [P1 §4-2 (the float packer), §1-1]
 *
 *   w       device [M][K] fp32, 16-byte aligned.
 *   packed  device [M][K/4] I2_S output, 16-byte aligned.
 *   w_max   HOST pointer or NULL; receives max |w| (0 for M == 0).
 *
 * Synchronises `stream`; M == 0 is a no-op.  Non-finite weights ->
 * BITNET_E_VALUE (packed then unspecified).
 */
int bitnet_pack_i2s_f32(const float *w, int64_t M, int64_t K, uint8_t *packed,
                        float *w_max, void *stream);

/*
 * bitnet_block_norm_quant_i8 -- the boundary between two blocks of a layer: the
 * norm after the block, its gate and residual scale, the residual stream, the
 * norm before the next block, and the tokens for that block's matmuls.
 * [P4 "Forward Pass"; P1 §4-5]
 *
 *   b        [N][F] the block's output (e.g. a projection's y), fp32 or bf16
 *            (b_dtype).
 *   post     non-zero: norm b first, with the gain post_gamma [F] or 1 (NULL).
 *   gate     fp32 or NULL (1): token n's row at gate + n * gate_stride;
 *            gate_stride is 0 (one row for every token) or at least F.
 *   scale    the residual scale, finite (1 for none).
 *   res, h   [N][F] the residual stream before and after, fp32 or bf16 (dtype).
 *            res NULL: no residual, h must be NULL.  h NULL: not stored.  h may
 *            be res itself; no other two arrays may overlap.
 *   gamma    [F] fp32 gain of the norm before the next block, or NULL for 1.
 *   eps      both norms' epsilon (positive, finite).
 *   v        [N][F] the normed tokens, in dtype, or NULL.
 *   xq, x_scale, x_sum   the tokens as bitnet_quant_act_i8 writes them, ready
 *            for the matmul calls; all three or none (NULL).
 *   At least one of h, v and xq is required.  F as K of the matmuls; rows and
 *   gains 16-byte aligned.  0 <= N < 2^31; N == 0 is a no-op.
 *
 * Per token, every operation one fp32 rounding and in this order:
 *   t = b;  post: t = (t * c) * post_gamma;  t = t * gate;  t = t * scale;
 *   with res: h = res + t, rounded to dtype, and the norm reads h as stored;
 *   v = (h * c) * gamma;  xq, x_scale, x_sum = bitnet_quant_act_i8 of v in fp32
 * where c = fp32(1 / sqrt(ss / F + eps)), ss the sum of the F squares in
 * binary64 (each square exact; one fixed order, which depends on F alone).
 * Non-finite inputs give unspecified results.
 */
int bitnet_block_norm_quant_i8(const void *b, int b_dtype, int post, const float *post_gamma,
                               const float *gate, int64_t gate_stride, float scale,
                               const void *res, void *h, int dtype, const float *gamma,
                               float eps, int64_t N, int64_t F, void *v, int8_t *xq,
                               float *x_scale, int32_t *x_sum, void *stream);

/*
 * The 4-bit key/value cache, and the sequences of a call.
 *
 * The cache is n_pages pages of BITNET_KV4_PAGE tokens; a page is n_kv_heads
 * records of 72 * head_dim bytes (4.5 bits a value).  head_dim is 64, 128 or
 * 256.  The memory is the caller's; it needs no initialisation, and what no
 * token was written to is never used.  Position p of sequence b is at token
 * p % 64 of page table[b][p / 64].  A table entry outside [0, n_pages) marks an
 * absent page: its tokens are not written, read as zeros and are not attended.
 *
 * A call's rows are tokens in order of their sequences: sequence b has the rows
 * [q_start[b], q_start[b + 1]), and they are its LAST positions: row q_start[b]
 * + i is at position kv_len[b] - (q_start[b + 1] - q_start[b]) + i.  So a step
 * adds its new tokens to kv_len and then passes the same q_start to the append
 * and the attention call.  q_start must not decrease, and all its rows lie in
 * [0, N).  Rows in front of q_start[0] and behind q_start[n_seqs] are neither
 * read nor written.  A row whose position is negative is not written, reads as
 * zeros and attends to nothing.  kv_len is held to [0, 64 * max_pages].
 *
 * A value is quantised with the 63 others of its token's group of 64 channels
 * (every operation one fp32 rounding):
 *   x is held to [-57344, 57344] (a NaN counts as -57344); lo, hi the group's ends
 *   mid  = fp16(lo + (hi - lo) * fp32(8/15))
 *   step = fp16(max((hi - mid) * fp32(1/7), (mid - lo) / 8))
 *   code = clamp(round_half_even((x - mid) * fp32(1/step) + 8), 0, 15); 8 if step is 0
 *   the value it stands for: mid + step * (code - 8)
 * The record: key codes [64 tokens][4][head_dim/32] dwords, dword (i, j) with
 * channels 32 j + 8 i + 0..7, the first in its low bits; value codes [16][16]
 * [head_dim/64][4] halfwords, halfword (a, i, g, t) with channels 64 g + 4 i +
 * 0..3 of token 4 a + t; key pairs [64][head_dim/64] (step, mid); value pairs
 * [16][head_dim/64] (4 steps, 4 mids) of four tokens.
 *
 *   table    [n_seqs][max_pages]   kv_len [n_seqs]   q_start [n_seqs + 1]
 * are DEVICE int32 arrays, read when the call's kernels run, so a captured call
 * follows their contents.  The descriptor itself is read during the call only.
 */
typedef struct {
    void *cache;            /* 16-byte aligned */
    int64_t n_pages;        /* 1 .. 2^31-1 */
    int64_t n_kv_heads;     /* 1 .. BITNET_KV4_MAX_HEADS */
    int64_t head_dim;       /* 64, 128 or 256 */
    const int32_t *table;
    int64_t max_pages;      /* 1 .. BITNET_KV4_MAX_PAGES */
    const int32_t *kv_len;
    const int32_t *q_start;
    int64_t n_seqs;         /* 0 .. BITNET_KV4_MAX_SEQS */
} bitnet_kv4_batch;

/*
 * bitnet_kv4_append -- quantise the keys and values of a call's rows into the
 * cache.
 *
 *   k, v     rows of n_kv_heads * head_dim fp32 or bf16 values, row n at k + n *
 *            k_stride elements (16-byte aligned, as the strides in bytes; a
 *            stride of at least a row, so slices of one merged projection do).
 *   0 <= N <= BITNET_GEMM_MAX_N; N == 0 or n_seqs == 0 is a no-op.
 * The cache overlaps neither k nor v, nor any call's outputs or workspace.
 * If two rows have the same place (one page in two sequences' tables), what
 * that token holds afterwards is unspecified; other tokens are not touched.
 */
int bitnet_kv4_append(const bitnet_kv4_batch *batch, const void *k, int64_t k_stride,
                      const void *v, int64_t v_stride, int dtype, int64_t N, void *stream);

/*
 * bitnet_kv4_read -- what the cache holds at a call's rows, as fp32 or bf16
 * (the fp32 value rounded to nearest even).
 *
 *   k, v     [N][n_kv_heads][head_dim] outputs, 16-byte aligned; one may be NULL.
 */
int bitnet_kv4_read(const bitnet_kv4_batch *batch, void *k, void *v, int dtype, int64_t N,
                    void *stream);

/*
 * bitnet_attn_kv4 -- causal attention of a call's rows over the cache, for
 * single tokens and prompts alike; the rows' own tokens are appended first.
 *
 *   q        rows of n_heads * head_dim fp32 or bf16 values, as k of the append;
 *            n_heads a multiple of n_kv_heads, head h reads kv head
 *            h / (n_heads / n_kv_heads).
 *   scale    of q . k, positive and finite (usually 1 / sqrt(head_dim)).
 *   window   0: a row at position p sees the positions 0 .. p; else those above
 *            p - window and the first `sinks` positions.
 *   max_kv   the longest kv_len that is expected (at most 64 * max_pages): it
 *            decides how many workgroups share a sequence and so the workspace
 *            and the speed, not what is computed.
 *   out      [N][n_heads][head_dim] in dtype, 16-byte aligned.  A row (one token,
 *            one head) that sees nothing gets zeros; one whose q has a NaN or an
 *            infinity is all NaN if it sees anything, and no other row is.
 *   workspace   device scratch of at least bitnet_attn_kv4_workspace bytes of the
 *            same sizes, 16-byte aligned (may be NULL where that is 0); used until the
 *            call's kernels have ended, so calls that may run at once need one
 *            each.
 *   0 <= N <= BITNET_GEMM_MAX_N; N == 0 or n_seqs == 0 is a no-op.  Calls of 2^24 or
 *   more workgroups are refused, by bitnet_attn_kv4_workspace (-1) too: none with
 *   N * n_heads / 16 + n_seqs * n_kv_heads below 2^24 is.
 *
 * Sums and maxima are fp32.  The softmax weights and their products with the
 * cache's steps are carried in 22 bits by fp32 calls (q too) and in 11 by bf16
 * calls, and no finer than 2^-27 (bf16: 2^-22) of a token's |mid| + 8 step at the
 * row's largest weight.  Rows whose |q| or scaled scores reach 2^100 are
 * unspecified.
 * Repeated calls with the same sizes give identical bits.
 */
int64_t bitnet_attn_kv4_workspace(int64_t n_seqs, int64_t N, int64_t n_heads,
                                  int64_t n_kv_heads, int64_t head_dim, int64_t max_kv,
                                  int64_t window, int64_t sinks);

int bitnet_attn_kv4(const bitnet_kv4_batch *batch, const void *q, int64_t q_stride, int dtype,
                    int64_t N, int64_t n_heads, float scale, int64_t window, int64_t sinks,
                    int64_t max_kv, void *out, void *workspace, int64_t workspace_bytes,
                    void *stream);

/*
 * Rotary positions.  Pair i of the first `rot` channels of a head's row, at position
 * p, is turned by 2 pi frac(p * turns[i] / 2^64):
 *   c = fp32(magnitude * cos), s = fp32(magnitude * sin)   (both from binary64)
 *   (a, b) -> (fl(fl(a c) - fl(b s)), fl(fl(b c) + fl(a s))), rounded to the row's type;
 * the other channels are copied.  turns[i] is the pair's frequency, in turns per position
 * as a 64-bit fraction of one (base^(-2 i / rot) / (2 pi) * 2^64, say, or any other by
 * which positions are scaled), so far positions lose nothing.
 */
typedef struct {
    const int64_t *turns;   /* DEVICE [rot / 2], 8-byte aligned */
    int64_t rot;            /* even, 2 .. head_dim */
    int interleaved;        /* 0: pairs (i, i + rot/2); else (2 i, 2 i + 1) */
    double magnitude;       /* positive and finite, below 1e30; 1 turns only */
} bitnet_rotary_plan;

/*
 * bitnet_rotary -- rows at given positions.
 *
 *   x        rows of n_heads * head_dim fp32 or bf16 values, row n at x + n * x_stride
 *            elements (16-byte aligned, as the strides in bytes; a stride of at least a
 *            row); head_dim a multiple of 8, at most BITNET_ROTARY_MAX_DIM.
 *   positions   DEVICE [N] int32 (negative ones turn the other way).
 *   inverse  non-zero: by the negative angle (the magnitude the same), which is the
 *            gradient of the forward call: dx from dout.
 *   out      as x; it may be x itself with the same stride, and overlaps it in no
 *            other way.
 *   1 <= n_heads <= BITNET_KV4_MAX_HEADS, 0 <= N <= BITNET_GEMM_MAX_N; N == 0 is a no-op.
 * A row with a NaN or an infinity has it, or a NaN, in the pair's two channels.
 */
int bitnet_rotary(const bitnet_rotary_plan *plan, const void *x, int64_t x_stride, int dtype,
                  int64_t N, int64_t n_heads, int64_t head_dim, const int32_t *positions,
                  int inverse, void *out, int64_t out_stride, void *stream);

/*
 * bitnet_rotary_kv4_append -- the step between a layer's projections and its attention in
 * one launch: q turned, k turned and appended to the cache, v appended.
 *
 *   batch, k, v   as bitnet_kv4_append.
 *   q, q_out      rows of n_heads * head_dim values as k; q_out may be q itself with the same
 *                 stride, and overlaps nothing else.  Rows of no sequence are left as they are.
 *   offset        DEVICE [n_seqs] int32 or NULL (0): a row at place p of the cache (see
 *                 above) has the position p + offset[b], e.g. where tokens were evicted.
 *   n_heads as bitnet_attn_kv4.
 * The results are bitnet_rotary's of q and k and bitnet_kv4_append's of what that gives, bit
 * for bit.
 */
int bitnet_rotary_kv4_append(const bitnet_kv4_batch *batch, const bitnet_rotary_plan *plan,
                             const void *q, int64_t q_stride, void *q_out, int64_t out_stride,
                             int64_t n_heads, const void *k, int64_t k_stride, const void *v,
                             int64_t v_stride, int dtype, int64_t N, const int32_t *offset,
                             void *stream);

/*
 * Matrices of 4-bit weights, for what a ternary model keeps finer than ternary (its output
 * head, its embedding).  A weight is step * (code - 8): a code of 4 bits each, a step (fp16,
 * of either sign) for each row and group of 32, 64 or 128 channels.
 *
 * Rows lie in tiles of 16 (rows behind the last are zeros), channels in blocks of 128, codes
 * as dwords of 8 channels, the first in the low bits:
 *   codes  [ceil(M/16)][K/128][4 quads][16 rows][4] dwords: dword (quad, row, j) has the
 *          block's channels 32 j + 8 quad + 0..7
 *   steps  [ceil(M/16)][K/128][16 rows][128/group] fp16, or with BITNET_W4_BY_GROUP
 *          [ceil(M/16)][K/128][128/group][16 rows]
 */
typedef struct {
    void *codes;            /* DEVICE, 16-byte aligned, ceil(M/16) * 8 * K bytes */
    void *steps;            /* DEVICE, 16-byte aligned, ceil(M/16) * 32 * K / group bytes */
    int64_t M;              /* 0 .. BITNET_W4_MAX_ROWS */
    int64_t K;              /* as K of the other matmuls */
    int64_t group;          /* 32, 64 or 128, plus BITNET_W4_BY_GROUP for steps in that order */
} bitnet_w4_matrix;

/*
 * bitnet_pack_w4 -- weights quantised into `mat`, group by group (every operation one
 * fp32 rounding):
 *   w is held to [-458528, 458528] (a NaN counts as 0); lo, hi the group's ends
 *   step = fp16(max(hi * fp32(1/7), -lo / 8))   (a zero is +0)
 *   code = clamp(round_half_even(w * fp32(1/step)), -8, 7) + 8; 8 if step is 0
 *
 *   w        [M][K] fp32 or bf16, 16-byte aligned.
 *
 * bitnet_pack_w4_codes -- weights that are 4-bit already: w [M][K] int8 in -8 .. 7 (held to
 * that), 8-byte aligned, and their steps given [M][K/group] fp16, 2-byte aligned.
 *
 * Both only enqueue.  M == 0 is a no-op.
 */
int bitnet_pack_w4(const void *w, int dtype, const bitnet_w4_matrix *mat, void *stream);
int bitnet_pack_w4_codes(const int8_t *w, const void *given, const bitnet_w4_matrix *mat,
                         void *stream);

/*
 * bitnet_w4_rows -- rows of the matrix as fp32 or bf16 (the fp32 value rounded to nearest even):
 * an embedding's lookup, or the weights read back.
 *
 *   ids      DEVICE [n] int32 row numbers, or NULL for rows 0 .. n-1.  One outside [0, M)
 *            gives zeros.
 *   out      [n][K], 16-byte aligned.  0 <= n <= BITNET_GEMM_MAX_N.
 */
int bitnet_w4_rows(const bitnet_w4_matrix *mat, const int32_t *ids, int64_t n, void *out,
                   int dtype, void *stream);

/*
 * bitnet_linear_w4 -- y[n][m] = sum_k x[n][k] * weight[m][k], for one token and for many.
 *
 *   x        [N][K] fp32 or bf16, 16-byte aligned.
 *   y        [N][M] fp32, 4-byte aligned.
 *   workspace   device scratch of at least bitnet_linear_w4_workspace bytes (-1: sizes out
 *            of range) of the same sizes, 16-byte aligned (may be NULL where that is 0); used
 *            until the call's kernels have ended, so calls that may run at once need one each.
 *   0 <= N <= BITNET_GEMM_MAX_N; N == 0 or M == 0 is a no-op.
 * A token's channels are carried in 22 bits (fp32; bf16 exactly) and no finer than 2^-40 of
 * the largest of their 128 (bf16: 2^-39); products and sums are fp32, so where the sum of
 * |x * weight| reaches 2^127 the result is unspecified.  A token with a NaN
 * or an infinity gives unspecified results, in its own row only.  Repeated calls give
 * identical bits.
 */
int64_t bitnet_linear_w4_workspace(int64_t N, int64_t M, int64_t K);

int bitnet_linear_w4(const void *x, int dtype, int64_t N, const bitnet_w4_matrix *mat, float *y,
                     void *workspace, int64_t workspace_bytes, void *stream);

/*
 * What attention weighed the cache's tokens with, and eviction by it.  A token's weight in a kv
 * head is one fp32 number; weights lie beside the cache as [n_pages][n_kv_heads]
 * [BITNET_KV4_PAGE] in the caller's memory, 16-byte aligned, and need no initialisation.
 *
 * bitnet_kv4_weigh -- adds the softmax weights of a call's rows to the tokens they see:
 *   out[t] = (t before the sequence's first row ? decay * weights[t] : 0)
 *            + the sum over its rows, and the heads that share the kv head, of p_t
 * for every position t < kv_len of each sequence that has rows in the call, on a page that
 * is there; nothing else of out is written.  The rows' own tokens begin at 0, so what was in
 * memory does not matter.  p are the weights of bitnet_attn_kv4 with the same arguments; the
 * call does not need its results and may run before or after it.
 *
 *   batch, q, q_stride, dtype, N, n_heads, scale, window, sinks, max_kv   as bitnet_attn_kv4.
 *   decay    finite, not negative; with 0 the weights are not read (NULL will do).
 *   out      may be weights itself, and overlaps them in no other way.
 *   workspace   device scratch of at least bitnet_kv4_weigh_workspace bytes (-1: sizes out
 *            of range) of the same sizes, 16-byte aligned; used until the call's kernels have
 *            ended, so calls that may run at once need one each.
 * A row that sees nothing or whose q has a NaN or an infinity adds nothing.  Where two
 * sequences with rows have one page, its weights are unspecified.  q is carried in 22 bits
 * (fp32; bf16 exactly), all else in fp32 (a p below 2^-126 of the row's largest may count as
 * 0); rows whose |q| or scaled scores reach 2^100 are
 * unspecified.  Repeated calls with the same sizes give identical bits.
 * One form of launch is taken for the whole call, by the rows of a sequence on average: long
 * chunks are quicker in a call of their own than in one with many single tokens.
 */
int64_t bitnet_kv4_weigh_workspace(int64_t n_seqs, int64_t N, int64_t n_heads, int64_t n_kv_heads,
                                   int64_t head_dim, int64_t max_kv, int64_t window,
                                   int64_t sinks);

int bitnet_kv4_weigh(const bitnet_kv4_batch *batch, const void *q, int64_t q_stride, int dtype,
                     int64_t N, int64_t n_heads, float scale, int64_t window, int64_t sinks,
                     int64_t max_kv, const float *weights, float decay, float *out, void *workspace,
                     int64_t workspace_bytes, void *stream);

/*
 * bitnet_kv4_evict -- copies what is kept of each sequence to the pages of another table.
 * Of the tokens at positions below kv_len whose page is there, min(their number, keep) are
 * kept, in each kv head its own: the first `sinks` positions, the last `recent` ones, and
 * of the others those of the largest weight (a NaN counts as -infinity; of equal ones the
 * first).  They stay in order and take the places 0, 1, ... of new_table, with their weights.
 * The old pages are left as they are.
 *
 *   batch       cache, table and kv_len; q_start is not looked at.
 *   weights     [n_pages][n_kv_heads][BITNET_KV4_PAGE], read at the old pages, written at
 *               the new ones.
 *   new_table   DEVICE [n_seqs][new_max_pages] int32, not table itself.  No page of it may be
 *               one that the call reads (of any sequence), or that it has twice: what they then
 *               hold is unspecified.  Tokens of a page that is absent in it are dropped.
 *   keep        1 .. 64 * new_max_pages; sinks and recent not negative, together at most keep.
 *   new_len     DEVICE [n_seqs] int32, other memory than kv_len: the number of tokens kept.
 *               (The rows' positions, which keys carry, do not change: the next row's is
 *               kv_len[b], not new_len[b], which is what the offsets of
 *               bitnet_rotary_kv4_append are for.)
 *   index       DEVICE [n_seqs][n_kv_heads][keep] int32: the position that each token had; -1
 *               behind the last.
 *   workspace   device scratch of at least bitnet_kv4_evict_workspace bytes (-1: sizes out
 *               of range) for these sizes, 16-byte aligned (may be NULL where that is 0); used
 *               until the call's kernels have ended, so calls that may run at once need one each.
 * A table of 320 pages or more is taken for one of long histories: of few sequences and heads it
 * has more launches, and a workspace.  n_seqs == 0 is a no-op.
 */
int64_t bitnet_kv4_evict_workspace(int64_t n_seqs, int64_t n_kv_heads, int64_t max_pages);

int bitnet_kv4_evict(const bitnet_kv4_batch *batch, float *weights, const int32_t *new_table,
                     int64_t new_max_pages, int64_t keep, int64_t sinks, int64_t recent,
                     int32_t *new_len, int32_t *index, void *workspace, int64_t workspace_bytes,
                     void *stream);

/* Thread-local description of the last non-OK status on this thread
 * (empty string if none).  The pointer stays valid until the next call on
 * the same thread. */
const char *bitnet_last_error(void);

/* BITNET_ABI_VERSION of the built library. */
int bitnet_abi_version(void);

#ifdef __cplusplus
}
#endif
#endif
