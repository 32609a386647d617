/*
 * kq.h - C ABI of libkq, the MI355X (gfx950) KroQuant online activation
 * quantizer.
 *
 * What it computes.  KroQuant (arXiv 2607.21446; read from the Pith review
 * page, "What carries the argument", core claim, and the referee report on
 * Sec. 3.2 Eqs. (4)-(6); and the AIssential summary page) quantizes the input
 * X[tokens][d] of a DiT linear layer to W4A4's activation side as follows:
 *   1. every 32-channel block j of a row is multiplied on the right by its
 *      own invertible 32x32 matrix K(j) = G1 (x) G2 (x) G3 (x) G4 (x) G5, a
 *      Kronecker product of five 2x2 unit-determinant LU factors
 *      G = [[1,0],[l,1]] [[a,b],[0,1/a]] = [[a, b], [l a, l b + 1/a]]
 *      (three scalars per factor, 15 per block); y = x K(j) in the
 *      row-vector convention of the review's Eq. (1);
 *   2. each transformed block of 32 is quantized to MXFP4 (OCP Microscaling
 *      Formats v1.0, the review's reference [10]): one E8M0 scale byte
 *      e + 127 with e = floor(log2 amax) - 2 (amax = 0 -> byte 0; clamped to
 *      [-127, 127]), and 32 E2M1 codes of y / 2^e rounded to nearest with
 *      ties to the even code and saturation at +-6; bit 3 of a code is the
 *      sign of y.
 * The pages compare this quantizer with a per-channel (SmoothQuant) scale and
 * a fixed Hadamard transform at the same block size (review, "If this is
 * right"; original abstract); those two, and a plain MXFP4 quantizer, are
 * here too with the same output format.
 *
 * Layouts (all row-major, little-endian):
 *   X         bf16 bit patterns [tokens][d], d a positive multiple of 32.
 *   K_params  fp32 [nb][5][3] (nb = d/32): (l, a, b) of G1 .. G5 for block j
 *             at K_params + j * params_block_stride (stride 15, or 0 for one
 *             K shared by every block).  a must be nonzero and finite.
 *   K_f32     fp32 [nb][32][32], K[r][c] (r = input channel, c = output).
 *   K_bf16    bf16 bit patterns [nb][n_split][32][32], TRANSPOSED: entry
 *             [j][s][c][r]; the terms hi = bf16(K), mid = bf16(K - hi),
 *             lo = bf16(K - hi - mid), each rounded to nearest even.  With
 *             three terms hi + mid + lo equals the fp32 K exactly.
 *   codes     uint8 [tokens][d/2]; byte q of block j holds the codes of
 *             channels 32j+2q (low nibble) and 32j+2q+1 (high nibble).
 *   scales    uint8 [tokens][d/32], E8M0 (2^(byte-127)).
 *   ch_mult   fp32 [d] per-channel multipliers (SmoothQuant: 1/s_c).
 *   Y         fp32 [tokens][d], the values the quantizer rounded.
 *
 * Numerics.  The transform runs in fp32 (fp32 butterfly stages, or MFMA bf16
 * products of X with a three-term bf16 split of K); the per-element error
 * against the exact sum is below 1e-5 of the block amax.  Whenever a
 * block's amax lands within 2^-16 (relative) of a power of two, the columns
 * that decide the scale are recomputed exactly (fp64 sum of exact products,
 * the fp32 K), so the E8M0 scales equal those of an exact evaluation.  An
 * E2M1 code can differ from the exact evaluation's only where y / 2^e lies
 * within that error of a rounding midpoint.  Plain and SmoothQuant
 * front-ends are exact.
 *
 * Ownership and streams.  The caller owns every buffer (device memory, e.g.
 * PyTorch tensors).  The library allocates nothing, frees nothing, keeps no
 * pointer after returning and never synchronizes: each call only enqueues
 * kernels on `stream` (NULL = the null stream) and returns.  Outputs must not
 * overlap inputs.  Reentrant and thread-safe; the only shared state is a
 * per-device cache of the compute-unit count, filled on first use.
 *
 * Errors.  Argument checks run before any HIP call and write nothing:
 *   KQ_ERR_NULL    a required pointer is NULL while tokens > 0;
 *   KQ_ERR_SHAPE   d <= 0, d % 32 != 0, d > 2^24, tokens < 0, tokens >= 2^28,
 *                  tokens * d >= 2^40,
 *                  nb <= 0, n_split not in 1..3, a stride other than 15 / 0;
 *   KQ_ERR_ALIGN   X, codes, Y, K_bf16, ch_mult not 16-byte aligned, or
 *                  K_params / K_f32 not 4-byte aligned;
 *   KQ_ERR_VARIANT unknown variant, or a variant whose inputs are missing
 *                  (KQ_MFMA_DENSE needs K_bf16; the others need K_params);
 *   KQ_ERR_ALIAS   an output range overlaps an input range or another output;
 *   KQ_ERR_WORKSPACE  a workspace is needed and NULL or too small.
 * tokens == 0 returns KQ_OK without touching the GPU.  A failed launch
 * returns KQ_ERR_HIP.  Faults inside a kernel surface at the caller's next
 * synchronization, as for any asynchronous HIP work.  No C++ exception
 * crosses this boundary.
 *
 * Interface notes (where these calls go beyond the plain form
 * kq_quantize(X, d, K_params, codes, scales, stream)):
 *   - every quantizing entry point takes `tokens`, the row count of X;
 *   - kq_quantize_ex takes no term count for K_bf16: KQ_MFMA_DENSE always
 *     reads the three-term split.  One bf16 term keeps 8 significant bits of
 *     each entry of K and two keep 16, so the transform error is bounded
 *     only by about 2^-9 or 2^-17 of sum_r |x_r K_rc|, which is above 1e-5
 *     of the block amax as soon as that sum exceeds 1.3 times the amax (as
 *     it does for most blocks); only three terms (the fp32 K exactly) keep
 *     the error within 1e-5 for every K.  kq_build_blocks still writes 1 to
 *     3 terms for other consumers;
 *   - kq_transform_f32 is one diagnostic entry for every front-end: it takes
 *     the front-end, the parameter stride, K_bf16 and ch_mult, and writes the
 *     codes and scales beside Y, so that each quantizing entry point's own
 *     kernel (plus a Y store) is what a test checks, codes included;
 *   - KQ_ERR_ALIAS: overlapping ranges are rejected with their own status
 *     rather than left undefined, since with an overlap the result would
 *     depend on the order in which the workgroups run.
 */
#ifndef KQ_H
#define KQ_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct ihipStream_t* hipStream_t;

typedef enum {
  KQ_OK = 0,
  KQ_ERR_NULL = 1,
  KQ_ERR_SHAPE = 2,
  KQ_ERR_ALIGN = 3,
  KQ_ERR_VARIANT = 4,
  KQ_ERR_HIP = 5,
  KQ_ERR_ALIAS = 6,
  KQ_ERR_WORKSPACE = 7
} kq_status;

/* How K is applied.  AUTO picks per shape: a kq_tune result if one was recorded, else the rule in kq_auto_variant. */
typedef enum {
  KQ_AUTO = 0,
  KQ_MFMA_DENSE = 1, /* MFMA bf16 contraction with prebuilt K_bf16 (three-term split) */
  KQ_MFMA_OTF = 2,   /* MFMA bf16 contraction, K rebuilt in-kernel from the 15 scalars */
  KQ_BUTTERFLY = 3   /* five fp32 butterfly stages (two shears each, then the product of the
                        diagonals) from the 15 scalars, one block per lane, no MFMA */
} kq_variant;

/* Front-ends of kq_transform_f32. */
typedef enum { KQ_FRONT_KRON = 0, KQ_FRONT_PLAIN = 1, KQ_FRONT_SMOOTH = 2, KQ_FRONT_HADAMARD = 3 } kq_front;

/* ABI version of this header (bumped on any signature or layout change). */
#define KQ_ABI_VERSION 8
int kq_abi_version(void);

/* Static, never-NULL description of a status code. */
const char* kq_status_str(kq_status status);

/*
 * Dense blocks from the 15 scalars per block (the "precomputed dense blocks"
 * kernel variant of the review, "What carries the argument").  For each of
 * nb blocks, with parameters at K_params + 15 j: K = G1 (x) ... (x) G5 with
 * every entry the product, in fp64 and in factor order, of one entry of each
 * factor (G1 on bit 4 of the row and column index, G5 on bit 0), then
 * rounded once to fp32.  Writes K_f32 [nb][32][32] if non-NULL and the
 * transposed bf16 split K_bf16 [nb][n_split][32][32] if non-NULL
 * (1 <= n_split <= 3).  At least one output must be non-NULL.
 */
kq_status kq_build_blocks(const float* K_params, int64_t nb, float* K_f32, uint16_t* K_bf16, int n_split,
                          hipStream_t stream);

/*
 * The online quantizer: codes and scales of X K for every block, with K
 * built from K_params (stride 15).  Equivalent to kq_quantize_ex(X, tokens,
 * d, K_params, 15, NULL, KQ_AUTO, out_codes, out_scales, stream).
 */
kq_status kq_quantize(const uint16_t* X, int64_t tokens, int64_t d, const float* K_params, uint8_t* out_codes,
                      uint8_t* out_scales, hipStream_t stream);

/*
 * As kq_quantize, choosing how K is applied.  params_block_stride is 15 (one
 * parameter set per block) or 0 (block 0's parameters, and K_bf16's block 0,
 * for every block).  K_bf16 (three-term split from kq_build_blocks, layout
 * above) is required by KQ_MFMA_DENSE and ignored by the other variants;
 * K_params is required by every variant except KQ_MFMA_DENSE.  KQ_AUTO uses
 * KQ_BUTTERFLY when K_params is given and KQ_MFMA_DENSE when only K_bf16 is
 * (unless kq_tune recorded another choice for the shape).
 */
kq_status kq_quantize_ex(const uint16_t* X, int64_t tokens, int64_t d, const float* K_params,
                         int64_t params_block_stride, const uint16_t* K_bf16, kq_variant variant,
                         uint8_t* out_codes, uint8_t* out_scales, hipStream_t stream);

/*
 * The variant KQ_AUTO resolves to for a call with this shape, given whether
 * K_params and K_bf16 are supplied (nonzero = supplied): the same rule the
 * entry points apply (a KQ_VARIANT override, else a kq_tune record, else
 * KQ_BUTTERFLY with K_params, KQ_MFMA_DENSE with K_bf16 alone).  Returns
 * KQ_AUTO when no variant can serve the call (neither input supplied).  Pure
 * host logic, no HIP call.
 *
 * Two environment variables, read once at the first call, exist for
 * measurement and change no result: KQ_VARIANT (mfma_dense, mfma_otf or
 * butterfly) replaces KQ_AUTO's choice wherever the supplied inputs allow
 * that variant, and KQ_WG_PER_CU (1 .. 64) caps the workgroups per compute
 * unit that every grid of the library is sized for.  Other values are ignored.
 */
kq_variant kq_auto_variant(int64_t tokens, int64_t d, int has_params, int has_split);

/* Plain MXFP4: y = x. */
kq_status kq_mx_quantize(const uint16_t* X, int64_t tokens, int64_t d, uint8_t* out_codes, uint8_t* out_scales,
                         hipStream_t stream);

/*
 * SmoothQuant front-end then MXFP4: y = fp32(x * ch_mult[c]) (one rounding),
 * the activation side of X diag(s)^-1 with ch_mult = 1/s (SmoothQuant, the
 * handbook page "Quantization: where diffusion differs from an LLM",
 * SmoothQuant section; the per-channel scaling baseline of the review).
 */
kq_status kq_smooth_quantize(const uint16_t* X, int64_t tokens, int64_t d, const float* ch_mult,
                             uint8_t* out_codes, uint8_t* out_scales, hipStream_t stream);

/*
 * Fixed block-Hadamard front-end then MXFP4: y[c] = fp32(sum_r x[r] H[r][c] /
 * sqrt(32)) with H[r][c] = (-1)^popcount(r & c) (natural-order Walsh-
 * Hadamard, orthonormal), the "fixed Hadamard at the same block size" of the
 * review's significance paragraph.
 */
kq_status kq_hadamard_quantize(const uint16_t* X, int64_t tokens, int64_t d, uint8_t* out_codes,
                               uint8_t* out_scales, hipStream_t stream);

/*
 * Block-Hadamard front-end of size `block` (32, 64, 128, 256 or 512; d a
 * multiple of it) then MXFP4 over blocks of 32: y[c] = fp32(sum_r x[r]
 * H[r][c] / sqrt(block)) within each block of `block` channels, the "larger
 * block sizes" a fixed Hadamard needs (Pith review, original abstract).
 * block = 32 is kq_hadamard_quantize.  Other sizes -> KQ_ERR_SHAPE.
 */
kq_status kq_hadamard_quantize_ex(const uint16_t* X, int64_t tokens, int64_t d, int block, uint8_t* out_codes,
                                  uint8_t* out_scales, hipStream_t stream);

/*
 * 16-wide KroQuant blocks with four factors (a block-size / factor-count
 * variant, 12 scalars per 16 channels at K_params16 + 12 b, (l, a, b) of
 * G1 .. G4, G1 on bit 3 of the 16-index): written as block-diagonal 32x32
 * blocks diag(K_{2j}, K_{2j+1}) in the layouts of kq_build_blocks (K_f32
 * [nb16/2][32][32], K_bf16 [nb16/2][n_split][32][32] transposed), each entry
 * the fp64 product in factor order rounded once to fp32, zeros off the
 * diagonal blocks.  Quantize with kq_quantize_ex(..., K_bf16, KQ_MFMA_DENSE).
 * nb16 must be even (KQ_ERR_SHAPE otherwise); errors as kq_build_blocks.
 */
kq_status kq_build_blocks16(const float* K_params16, int64_t nb16, float* K_f32, uint16_t* K_bf16, int n_split,
                            hipStream_t stream);

/*
 * Per-shape tuning of KQ_AUTO (opt-in).  Times the variant the built-in rule
 * picks and every variant the supplied inputs allow (KQ_MFMA_OTF and
 * KQ_BUTTERFLY need K_params with stride 15, KQ_MFMA_DENSE needs K_bf16), the
 * MFMA variants each with fourteen grid shapes (seven sizes of the second
 * part of the grid, the share of row tiles left to workgroups that start as
 * others finish and the tiles each of those takes, times a first part sized
 * for the resident workgroups per CU or for one; outputs do not depend on the
 * grid shape), on the caller's buffers: three interleaved rounds of 3 warm-up
 * launches and `reps` timed launches per candidate (1 <= reps <= 1000, else
 * KQ_ERR_SHAPE), timed with events on `stream`, each candidate scored by its
 * median round.  The fastest candidate is recorded if it is at least 3%
 * faster than the built-in rule's, else the rule's choice is (the timing
 * reuses one set of buffers, which can stay in the last-level cache; the
 * margin keeps a pick that only wins warm from replacing the rule).  The
 * record is keyed by (tokens, d, which inputs are supplied), process-wide:
 * later KQ_AUTO calls with that key use its variant (kq_auto_variant reports
 * it; a KQ_VARIANT environment override still wins), and later kq_quantize /
 * kq_quantize_ex calls with that key, stride 15 and that variant use its grid
 * shape.  On return out_codes / out_scales hold the recorded variant's result
 * and *chosen (if not NULL) the variant.  This is the one entry point that
 * blocks: it synchronizes on its timing event.  Neither input ->
 * KQ_ERR_VARIANT; other errors as kq_quantize_ex; a failed launch or event ->
 * KQ_ERR_HIP.
 */
kq_status kq_tune(const uint16_t* X, int64_t tokens, int64_t d, const float* K_params, const uint16_t* K_bf16,
                  uint8_t* out_codes, uint8_t* out_scales, int reps, kq_variant* chosen, hipStream_t stream);

/* Forget every choice kq_tune recorded (KQ_AUTO falls back to its default rule). */
void kq_tune_reset(void);

/*
 * Diagnostic entry (tests): runs the same kernels as the entries above and
 * also stores Y, the fp32 values each code was rounded from.  front selects
 * the front-end; variant, K_params, params_block_stride and K_bf16 apply to
 * KQ_FRONT_KRON as in kq_quantize_ex, ch_mult to KQ_FRONT_SMOOTH.
 */
kq_status kq_transform_f32(int front, const uint16_t* X, int64_t tokens, int64_t d, const float* K_params,
                           int64_t params_block_stride, const uint16_t* K_bf16, kq_variant variant,
                           const float* ch_mult, float* Y, uint8_t* out_codes, uint8_t* out_scales,
                           hipStream_t stream);

/*
 * LayerNorm statistics per row, for the AdaLN producer step below (the
 * normalisation without affine parameters that precedes a DiT linear
 * layer's AdaLN modulation; the Pith review's summary gives AdaLN as the
 * reason the transform runs online, its ledger lists LayerNorm / AdaLN as
 * normalisations that do not commute with it).  For each row t:
 *   mean = sum_c x / d, var = sum_c (x - mean)^2 / d   (fp64 sums),
 *   rstd = 1 / sqrt(var + eps)                         (fp64),
 * stored as fp32 row_stats[2t] = mean, row_stats[2t+1] = rstd.  The fp64
 * summation order is unspecified: results can differ from a sequential
 * evaluation by one fp32 ulp, rarely.  Errors as above; eps < 0 or not finite
 * -> KQ_ERR_SHAPE; X 16-byte and row_stats 8-byte aligned.
 */
kq_status kq_row_stats(const uint16_t* X, int64_t tokens, int64_t d, float eps, float* row_stats,
                       hipStream_t stream);

/*
 * The quantizer with the AdaLN producer step fused in front of the transform
 * (one read of X instead of a modulation kernel's read + write followed by
 * the quantizer's read).  Each element, in fp32, one IEEE operation each and
 * in this order (no contraction):
 *   v = x;
 *   v = (v - mean_t) * rstd_t                 if row_stats != NULL ([tokens][2], above);
 *   v = v * (1 + mod_scale[s][c])             if mod_scale != NULL;
 *   v = v + mod_shift[s][c]                   if mod_shift != NULL;
 * with s = t / tokens_per_sample and mod_scale, mod_shift fp32
 * [ceil(tokens / tokens_per_sample)][d]; v is rounded to bf16 (nearest even)
 * and then transformed and quantized exactly as kq_quantize_ex would
 * transform and quantize that bf16 matrix (the handbook page "Quantization:
 * where diffusion differs from an LLM" describes AdaLN as timestep-dependent
 * per-channel scales and shifts; the form v (1 + scale) + shift is the DiT
 * one).  tokens_per_sample must be a multiple of 32 or at least tokens
 * (KQ_ERR_SHAPE otherwise).  Variants as kq_quantize_ex, with the same
 * inputs and the same rule for KQ_AUTO: every variant applies the producer
 * step, and the codes and scales equal those kq_quantize_ex gives with that
 * variant on the modulated bf16 matrix, bit for bit.
 * row_stats must be 8-byte aligned, mod_scale / mod_shift 16-byte aligned
 * (KQ_ERR_ALIGN otherwise).
 */
kq_status kq_quantize_adaln(const uint16_t* X, int64_t tokens, int64_t d, const float* row_stats,
                            const float* mod_scale, const float* mod_shift, int64_t tokens_per_sample,
                            const float* K_params, int64_t params_block_stride, const uint16_t* K_bf16,
                            kq_variant variant, uint8_t* out_codes, uint8_t* out_scales, hipStream_t stream);

/*
 * Blocks of the offline weight fold (Pith review, circularity check:
 * Eq. (1), A T (W T^-T)^T = A W^T): as kq_build_blocks, for
 * K^-T = (G1^-1)^T (x) ... (x) (G5^-1)^T with G^-1 = [[l b + 1/a, -b],
 * [-l a, a]] (each entry the fp64 product in factor order, rounded once to
 * fp32; same layouts and errors).  The folded, quantized weight is then
 * kq_quantize_ex(W, N_out, K_in, NULL, 15, K_bf16 of these blocks,
 * KQ_MFMA_DENSE, w_codes, w_scales, stream) for a bf16 weight W [N_out][K_in]
 * (rows = output features), i.e. every weight row times T^-T, quantized to
 * MXFP4 along K_in.
 */
kq_status kq_build_blocks_inverse_t(const float* K_params, int64_t nb, float* K_f32, uint16_t* K_bf16, int n_split,
                                    hipStream_t stream);

/*
 * W4A4 GEMM on the scaled FP4 matrix cores: Y[m][n] = sum_k a[m][k] b[n][k]
 * with a = E2M1(code) * 2^(scale - 127) from A (codes [M][K/2], scales
 * [M][K/32], the layout kq_quantize writes) and b likewise from B [N][K]
 * (a folded weight from kq_build_blocks_inverse_t + kq_quantize_ex).  Each
 * product is exact; sums are fp32 (per element error below K 2^-24 sum|a b|
 * in practice).  Writes Y_f32 [M][N] fp32 and/or Y_bf16 [M][N] bf16 (nearest
 * even), either may be NULL but not both.  K a positive multiple of 32
 * (<= 2^24), M <= 2^23, N <= 2^22, else KQ_ERR_SHAPE; codes 16-byte aligned;
 * outputs must not overlap inputs.  M == 0 or N == 0 returns KQ_OK.
 */
kq_status kq_gemm_mx(const uint8_t* A_codes, const uint8_t* A_scales, int64_t M, const uint8_t* B_codes,
                     const uint8_t* B_scales, int64_t N, int64_t K, float* Y_f32, uint16_t* Y_bf16,
                     hipStream_t stream);

/* Activations of kq_gemm_mx_ex. */
typedef enum {
  KQ_ACT_NONE = 0,
  KQ_ACT_GELU_TANH = 1, /* x (1 + tanh(sqrt(2/pi) (x + 0.044715 x^3))) / 2 */
  KQ_ACT_GELU_ERF = 2,  /* x (1 + erf(x / sqrt 2)) / 2 */
  KQ_ACT_SILU = 3       /* x / (1 + exp(-x)) */
} kq_act;

/*
 * kq_gemm_mx with what a transformer layer does next on the fp32 sums, before
 * the one rounding of the output: with s = sum_k a[m][k] b[n][k],
 *   s = s + bias[n]                          if bias != NULL     (fp32 [N]);
 *   s = act(s);
 *   s = s * gate[m / rows_per_sample][n]     if gate != NULL     (fp32
 *                      [ceil(M / rows_per_sample)][N], the AdaLN gate);
 *   s = residual[m][n] + s                   if residual != NULL (bf16 [M][N]),
 * in fp32 and in this order (an activation's absolute error is below 2^-21
 * max(|x|, 1)).  Y_bf16 may be residual itself (the residual stream
 * updated in place); any other overlap is KQ_ERR_ALIAS.  rows_per_sample is
 * any positive number (KQ_ERR_SHAPE otherwise), read only with gate; an
 * unknown act is KQ_ERR_VARIANT; bias and gate 4-byte, residual 2-byte
 * aligned.  Otherwise as kq_gemm_mx; the sums may be formed in another order
 * than kq_gemm_mx's (few rows split K over the waves of a workgroup), always
 * the same one for the same sizes.
 */
kq_status kq_gemm_mx_ex(const uint8_t* A_codes, const uint8_t* A_scales, int64_t M, const uint8_t* B_codes,
                        const uint8_t* B_scales, int64_t N, int64_t K, const float* bias, kq_act act,
                        const float* gate, int64_t rows_per_sample, const uint16_t* residual, float* Y_f32,
                        uint16_t* Y_bf16, hipStream_t stream);

/*
 * Key/value cache in MXFP4.  A cache is four pools with n_slots rows each:
 * codes [n_slots][width/2] and E8M0 scales [n_slots][width/32] of keys and of
 * values, row-major, width = kv_heads * head_dim (a multiple of 32; the 32
 * channels of a block are consecutive in a row and may span two heads).  Row
 * s is slot s, in the format kq_mx_quantize writes: a cache whose slots are in
 * order can also be filled by any quantizer of this library.
 *
 * kq_cache_write quantizes rows t = 0 .. tokens - 1 of K (and of V, unless V
 * is NULL) as kq_mx_quantize does and writes them to slot slots[t].  A token
 * whose slot is outside [0, n_slots) (padding: -1) is not written; slots that
 * no token names keep their contents.  Slots are meant to be distinct: of two
 * tokens with the same slot either may be left there, block by block, codes
 * and scales not necessarily from the same one.
 *
 * kq_cache_read writes the values of slot slots[t] to row t of K (and V):
 * bf16(E2M1(code) * 2^(scale - 127)), exact for every scale this library
 * writes (0 .. 252; above that a value past the bf16 range is infinite, and
 * scale 255 reads as NaN).  A token whose slot is outside [0, n_slots) reads
 * as zeros.  Slots may repeat.
 *
 * K and V are bf16 rows at strides K_stride and V_stride (elements; a multiple
 * of 8, at least width), 16-byte aligned: columns of a wider matrix, such as a
 * fused projection's output, serve as they are.  Codes 16-byte, scales and
 * slots 4-byte aligned.  n_slots < 2^31; V's pools are not read when V is
 * NULL.  One launch for both.
 */
kq_status kq_cache_write(const uint16_t* K, int64_t K_stride, const uint16_t* V, int64_t V_stride, int64_t tokens,
                         int64_t width, const int32_t* slots, int64_t n_slots, uint8_t* K_codes, uint8_t* K_scales,
                         uint8_t* V_codes, uint8_t* V_scales, hipStream_t stream);

kq_status kq_cache_read(const uint8_t* K_codes, const uint8_t* K_scales, const uint8_t* V_codes,
                        const uint8_t* V_scales, int64_t n_slots, int64_t width, const int32_t* slots, int64_t tokens,
                        uint16_t* K, int64_t K_stride, uint16_t* V, int64_t V_stride, hipStream_t stream);

/*
 * Attention of bf16 queries over such a cache: for query i of a sequence and
 * query head h, with key head h / (q_heads / kv_heads),
 *   out = sum_j softmax_j(scale q.k_j) v_j,   lse = log sum_j exp(scale q.k_j)
 * over the keys j it sees.  The rule of precision: q, k and v enter the
 * products unrounded, scores, maxima and sums are fp32, the probabilities
 * (relative to the running maximum) are rounded once to bf16 before they
 * multiply v, the output is rounded once.
 *
 * Queries: Q and out are bf16 [q_rows] rows of q_heads * head_dim at strides
 * Q_stride and out_stride (elements, a multiple of 8), 16-byte aligned.
 * Sequence b has rows q_start[b] .. q_start[b + 1] - 1 (int32 [batch + 1],
 * not decreasing), or, with q_start NULL, rows b max_q .. (b + 1) max_q - 1.
 * max_q bounds the queries of a sequence (<= q_rows); queries past it are not
 * computed.  Ranges are cut to [0, q_rows).  Rows of out and lse that belong
 * to no sequence are left as they are.
 *
 * Keys: sequence b has kv_len[b] of them (int32; cut to [0, pages_per_seq *
 * page_size]).  Key j is at slot page_table[b][j / page_size] * page_size +
 * j % page_size (int32 [batch][pages_per_seq]; pages may be shared), or, with
 * page_table NULL, at slot b pages_per_seq page_size + j.  A key on a page
 * outside [0, n_slots / page_size) is not there: as if masked.  page_size is
 * any number from 1 to 2^24.  Nothing of a slot that no key names is used,
 * whatever it holds.  causal != 0: with n queries and L keys, query i sees
 * keys j <= L - n + i (the queries are the sequence's last tokens), else all
 * L.  A query that sees no key, or whose scores are all -infinity, gets out = 0
 * and lse = -infinity; a NaN among the scores of a query makes its out and
 * lse NaN.  A value that is not finite (scale bytes above 252, which only
 * tokens that were not finite get) may also reach queries of its sequence
 * that do not see its key.
 *
 * head_dim is a multiple of 8 from 8 to 128, q_heads a multiple of kv_heads,
 * scale positive and at most 2^127 (scale q.k itself has to stay within fp32,
 * as every score does).  lse (fp32 [q_rows][q_heads]) may be NULL.
 * Limits (KQ_ERR_SHAPE past them): q_rows < 2^28, batch and q_heads <= 65535,
 * batch * max_q * q_heads and pages_per_seq * page_size <= 2^30, n_slots <
 * 2^31, and less than 2^32 threads in a launch (65535 sequences of one query:
 * up to 255 key heads, 510 where a workgroup takes two).
 * Long key ranges with few queries, and of many queries those that the GPU
 * would compute last and not all at work, are divided over workgroups and
 * joined in a second launch; the partial results need kq_attention_mx_workspace bytes
 * (0: none, workspace may be NULL), 16-byte aligned, free again when the call
 * has run: calls that may run at the same time, two captured graphs among
 * them, need one each.  The division depends on the sizes and the lengths
 * alone, so the same call gives the same bits.  capacity = pages_per_seq * page_size.
 */
int64_t kq_attention_mx_workspace(int64_t q_rows, int64_t batch, int64_t max_q, int64_t q_heads, int64_t kv_heads,
                                  int64_t head_dim, int64_t capacity);

kq_status kq_attention_mx(const uint16_t* Q, int64_t Q_stride, int64_t q_rows, const int32_t* q_start, int64_t batch,
                          int64_t max_q, const uint8_t* K_codes, const uint8_t* K_scales, const uint8_t* V_codes,
                          const uint8_t* V_scales, int64_t n_slots, const int32_t* page_table, int64_t pages_per_seq,
                          int64_t page_size, const int32_t* kv_len, int64_t q_heads, int64_t kv_heads,
                          int64_t head_dim, float scale, int causal, uint16_t* out, int64_t out_stride, float* lse,
                          void* workspace, int64_t workspace_bytes, hipStream_t stream);

/* Norms over channels: none, x / sqrt(mean x^2 + eps), (x - mean) / sqrt(mean (x - mean)^2 + eps). */
typedef enum { KQ_NORM_NONE = 0, KQ_NORM_RMS = 1, KQ_NORM_LAYER = 2 } kq_norm;

/* Which channels of a head are pair p of the R/2 that turn: 2p and 2p + 1, or p and p + R/2. */
typedef enum { KQ_ROPE_PAIRS = 0, KQ_ROPE_HALVES = 1 } kq_rope_layout;

/*
 * Rotary positions with several axes (a token's place in a text; its time, row
 * and column in a video).  axis_dims[i] channels of each head (even, positive)
 * turn with axis i, the pairs of axis 0 first; R is their sum, at most
 * head_dim, and channels from R on do not turn.  Pair p of axis i turns by
 * positions[t][i] * freqs[p] radians.  This struct lies in host memory and is
 * read before the call returns; positions and freqs are device memory.  A NULL
 * rotation, or n_axes 0, turns nothing.
 */
typedef struct {
  const int32_t* positions; /* [tokens][n_axes] */
  const double* freqs;      /* [R/2], finite; an angle below 2^48 in size */
  int32_t n_axes;           /* 0 .. 4 */
  int32_t axis_dims[4];
  kq_rope_layout layout;
} kq_rotation;

/*
 * Rows of heads (queries, keys) normalised and turned: for each head of
 * head_dim channels (a multiple of 8, 8 .. 128) of row t
 *   n = x                                        norm KQ_NORM_NONE, or
 *   n = x weight / sqrt(mean(x^2) + eps)         KQ_NORM_RMS (weight fp32 [head_dim], NULL: 1);
 *   (u, v) of a pair -> (u cos a - v sin a, u sin a + v cos a),
 * rounded once to bf16 (below 2^-126 by way of fp32's last step, 2^-149):
 * everything before is fp64, the angles too, so far positions keep theirs (to
 * 2^-51 of the angle, and 2^-40).  X and out are bf16
 * [tokens][heads * head_dim] at strides X_stride and out_stride
 * (elements, a multiple of 8), 16-byte aligned; out may be X itself at the
 * same stride, or other columns of the same matrix; any other overlap is
 * KQ_ERR_ALIAS.  KQ_NORM_LAYER and unknown layouts are KQ_ERR_VARIANT; axes
 * that are odd, negative or more than head_dim together KQ_ERR_SHAPE, as are
 * more than 2^21 heads or 2^24 channels.  weight and positions 4-byte, freqs
 * 8-byte aligned.  A row of zeros with eps 0 is NaN, as the formula's.
 */
kq_status kq_rope(const uint16_t* X, int64_t X_stride, int64_t tokens, int64_t heads, int64_t head_dim, kq_norm norm,
                  const float* weight, float eps, const kq_rotation* rotation, uint16_t* out, int64_t out_stride,
                  hipStream_t stream);

/*
 * kq_cache_write of keys that are normalised and turned on the way, with the
 * queries of the same tokens turned in the same launch: K's heads as kq_rope
 * (with k_weight) and then, from that bf16, as kq_cache_write; V as
 * kq_cache_write (V may be NULL); Q, unless NULL, as kq_rope with q_weight
 * into Q_out.  The results equal those calls', bit for bit.  A token without a
 * slot still has its query turned.  kv_heads * head_dim is a multiple of 32;
 * q_heads is any positive number, read only with Q.  Q_out may be Q itself and
 * Q, K and V columns of one matrix: a fused projection's output can be
 * passed as it is and its queries turned in place.  Otherwise as kq_rope and
 * kq_cache_write.
 */
kq_status kq_cache_write_rope(const uint16_t* Q, int64_t Q_stride, int64_t q_heads, const float* q_weight,
                              uint16_t* Q_out, int64_t Q_out_stride, const uint16_t* K, int64_t K_stride,
                              const uint16_t* V, int64_t V_stride, int64_t tokens, int64_t kv_heads, int64_t head_dim,
                              kq_norm norm, const float* k_weight, float eps, const kq_rotation* rotation,
                              const int32_t* slots, int64_t n_slots, uint8_t* K_codes, uint8_t* K_scales,
                              uint8_t* V_codes, uint8_t* V_scales, hipStream_t stream);

/*
 * The residual stream between two blocks: what a block gave (Y) is normalised
 * and gated and added to the stream X, and the next block's input is taken
 * from the sum.  Per row t of sample s = t / tokens_per_sample:
 *   u  = N_post(y) * post_weight * gate[s]             post_weight fp32 [d], gate fp32 [samples][d], each may be NULL
 *   x' = residual_scale * x + u                        -> X_out, bf16
 *   h  = N_pre(x') * pre_weight * (1 + mod_scale[s]) + mod_shift[s]
 *                                                      -> H, bf16, and / or out_codes and out_scales, as
 *                                                         kq_mx_quantize of that bf16 matrix, and / or
 *   row_stats[t] = (mean, 1 / sqrt(var + eps)) of x'   fp32, as kq_row_stats (mean 0 for KQ_NORM_RMS): what
 *                                                      kq_quantize_adaln reads to transform and quantize x'
 * with the norms of kq_norm over the row's d channels, statistics of x' taken
 * from the bf16 values that are stored, and samples = ceil(tokens /
 * tokens_per_sample).  Arithmetic and sums are fp64 up to each rounding
 * (roundings to bf16 as kq_rope's); a channel that equals its row's mean is 0
 * after a layer norm.  Statistics may differ from kq_row_stats' by an fp32
 * step, where a sum lies next to a tie.  h is rounded once, so it may differ by
 * a bf16 step from what kq_quantize_adaln forms in fp32 steps.
 *
 * Y NULL: the stream is X as it is (x' = x, the first block's norm): X_out,
 * post, post_weight, gate have to be NULL / KQ_NORM_NONE and residual_scale 1
 * (KQ_ERR_VARIANT otherwise).  With Y, X_out is needed and H, codes and
 * statistics may all be NULL.  out_codes and out_scales come together.
 * row_stats needs a norm (KQ_ERR_VARIANT).  tokens_per_sample is any positive
 * number, read with gate, mod_scale or mod_shift.
 *
 * X, Y, X_out and H are rows at strides in elements (a multiple of 8, at least
 * d; d a multiple of 32), 16-byte aligned, vectors 16-byte, row_stats 8-byte
 * aligned.  X_out may be X itself at the same stride (the stream updated in
 * place); rows may be columns of one matrix that do not touch; any other
 * overlap is KQ_ERR_ALIAS.  eps >= 0 and residual_scale finite
 * (KQ_ERR_SHAPE).
 */
kq_status kq_residual_norm(const uint16_t* X, int64_t X_stride, const uint16_t* Y, int64_t Y_stride, int64_t tokens,
                           int64_t d, kq_norm post, const float* post_weight, const float* gate, float residual_scale,
                           uint16_t* X_out, int64_t X_out_stride, kq_norm pre, const float* pre_weight,
                           const float* mod_scale, const float* mod_shift, int64_t tokens_per_sample, float eps,
                           uint16_t* H, int64_t H_stride, uint8_t* out_codes, uint8_t* out_scales, float* row_stats,
                           hipStream_t stream);

/*
 * Measurement entry (not a quantizer): moves exactly the traffic of
 * kq_quantize's default kernel on X [tokens][d] (every bf16 of X read once in
 * 4 KB units of 64 consecutive 32-channel blocks, one 16-byte record per
 * block written to out_codes [tokens][d/2] and one byte per block to
 * out_scales [tokens][d/32], each wave's units in the same order, through the
 * same wave-private LDS round trip; the grid is sized for the probe's own
 * occupancy, one resident round of waves) with no arithmetic:
 * the outputs hold an XOR digest of the input, not codes.  Its rate is the
 * ceiling this access pattern reaches on the device, against which the
 * quantizers' rates are reported (the Pith review's Fig. 3 reports the
 * quantizer's effective HBM bandwidth).  Errors as kq_mx_quantize.
 */
kq_status kq_stream_probe(const uint16_t* X, int64_t tokens, int64_t d, uint8_t* out_codes, uint8_t* out_scales,
                          hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* KQ_H */
