/*
 * fp8q.h -- C ABI of libfp8q: fine-grained FP8 (E4M3) quantisation and the
 * per-group-scaled FP8 GEMM on one sm_103a GPU.
 *
 * The operations follow the FP8 training recipe of DeepSeek-V3 as described
 * on these pages:
 *   - dssusan.co.kr board post 91437 (an excerpt of the DeepSeek-V3 report's
 *     FP8 section): paragraph 1 (power-of-two scaling factors for some
 *     activations), paragraph 2 (max-abs computed online per 1x128 activation
 *     tile and per 128x128 weight block; the scaling factor follows from it),
 *     paragraph 3 (Figure 6: per-group scaling factors along the GEMM's inner
 *     dimension K, applied as dequantisation, FP32 accumulation), paragraph 4
 *     (Figure 7 (a): 1x128 per token per 128 channels, 128x128 per 128 input
 *     by 128 output channels; 1x128 tiles become 128x1 tiles in the backward
 *     pass);
 *   - "Deepseek - Not For everyone" (xn--jj0bz6z98ct0a29q.com post 278251),
 *     paragraph 4: the max-abs is mapped onto the largest finite FP8 value;
 *   - youlimart.com FAQ post 597629, paragraph 2 (Figure 6): Fprop, Dgrad and
 *     Wgrad all run in FP8, taking FP8 inputs and producing BF16 or FP32;
 *   - "FP8 mixed precision -- где и как DeepSeek снизили точность
 *     вычислений?" (Data Science by ODS.ai): E4M3 for every tensor, FP32
 *     accumulation of the tensor-core partial sums.
 *
 * Conventions for every call:
 *   - Tensors are row-major; every leading dimension (ld*) is in ELEMENTS of
 *     that tensor's type.  E4M3 tensors are raw bytes (1 byte per element),
 *     BF16 tensors raw 16-bit patterns.
 *   - All pointers are DEVICE pointers owned by the caller; the library never
 *     allocates or frees device memory, and keeps none of the caller's
 *     pointers after a call returns (the only device address it keeps is that
 *     of its own static scratch array, see fp8q_quant_tensor_noalloc).  Calls
 *     are asynchronous on `stream` (a cudaStream_t; NULL is the legacy
 *     default stream).
 *   - E4M3 means the OCP "E4M3FN" encoding (bias 7, largest finite 448, NaN
 *     0x7F/0xFF, no infinity).  Values are rounded to nearest-even and
 *     saturated to +-448.
 *   - Scales s are FP32 with dequantised value = decode(q) * s.  For a group
 *     with max-abs value amax, a = max(amax, 2^-116) and
 *       FP8Q_SCALE_FP32: s = a / 448, codes E4M3(x * (448 / a)), both FP32
 *                        divisions rounded to nearest;
 *       FP8Q_SCALE_POW2: s = 2^e, e the smallest integer with 448 * 2^e >= a,
 *                        codes E4M3(x * 2^-e).
 *     Inputs must be finite; NaN/Inf inputs give unspecified codes.
 *   - Argument errors are returned synchronously and nothing is launched.
 *     A device-side failure (a bounded wait that gave up) is recorded in a
 *     device status word and returned by fp8q_sync_status().
 */
#ifndef FP8Q_H
#define FP8Q_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum fp8q_status {
  FP8Q_OK = 0,
  FP8Q_ERR_INVALID = 1,     /* null pointer where one is required, unknown enum */
  FP8Q_ERR_SHAPE = 2,       /* negative size, K/T not a multiple of 128, ld too small */
  FP8Q_ERR_ALIGN = 3,       /* pointer or leading dimension breaks a 16-byte rule */
  FP8Q_ERR_UNSUPPORTED = 4, /* current device is not sm_103, or too little shared memory */
  FP8Q_ERR_CUDA = 5,        /* a CUDA runtime call or kernel launch failed */
  FP8Q_ERR_TIMEOUT = 6      /* a device-side wait gave up (reported by fp8q_sync_status) */
} fp8q_status;

enum { FP8Q_SCALE_FP32 = 0, FP8Q_SCALE_POW2 = 1 };
enum { FP8Q_OUT_BF16 = 0, FP8Q_OUT_FP32 = 1 };
/* Layout of the B-operand scales of fp8q_gemm. */
enum {
  FP8Q_BSCALE_BLOCK = 0,   /* one per 128x128 block:  sb[(n/128) * ld_sb + k/128] */
  FP8Q_BSCALE_BLOCK_T = 1, /* one per 128x128 block, grid transposed:
                              sb[(k/128) * ld_sb + n/128] (Dgrad reading a weight's grid) */
  FP8Q_BSCALE_ROW = 2      /* one per row n per 128-K group (128x1 tiles, Wgrad):
                              sb[(k/128) * ld_sb + n] */
};

/*
 * Activation quantisation, 1x128 tiles: one scale per row (token) m per 128
 * columns (channels) ([dssusan] paragraph 2 and paragraph 4, Figure 7 (a)(1)).
 *   x   BF16 [M][ldx], reads columns [0, K).       K % 128 == 0, M >= 0.
 *   q   E4M3 [M][ldq], writes columns [0, K).
 *   sa  FP32, MN-major: scale of (m, group g) at sa[g * ld_sa + m], ld_sa >= M.
 * Alignment: x and q 16-byte aligned, ldx % 8 == 0, ldq % 16 == 0.
 */
fp8q_status fp8q_quant_act(const void *x, int64_t M, int64_t K, int64_t ldx,
                           void *q, int64_t ldq, float *sa, int64_t ld_sa,
                           int scale_mode, void *stream);

/*
 * Activation quantisation for the backward pass, 128x1 tiles: one scale per
 * column (channel) c per 128 rows (tokens) ([dssusan] paragraph 4: 1x128
 * tiles become 128x1 tiles).  The codes are written TRANSPOSED so the token
 * dimension is contiguous, i.e. K-major for the Wgrad GEMM.
 *   x      BF16 [T][ldx], columns [0, C).           T % 128 == 0, C % 8 == 0,
 *          T <= 65535 * 128, C <= 2^31 - 128 (else FP8Q_ERR_SHAPE).
 *   qT     E4M3 [C][ldqT], qT[c][t] = code of x[t][c].
 *   sT     FP32, scale of (t-group tg, c) at sT[tg * ld_sT + c], ld_sT >= C.
 *   q_rows optional (NULL to skip): the 1x128 quantisation of the same x,
 *          computed from the same read: E4M3 [T][ldq_rows] and
 *          s_rows[g * ld_s_rows + t] exactly as fp8q_quant_act would write
 *          them.  Requires C % 128 == 0; s_rows must then be non-NULL.
 * Alignment: x, qT (and q_rows) 16-byte aligned; ldx % 8, ldqT % 16,
 * ldq_rows % 16 == 0.
 */
fp8q_status fp8q_quant_act_T(const void *x, int64_t T, int64_t C, int64_t ldx,
                             void *qT, int64_t ldqT, float *sT, int64_t ld_sT,
                             void *q_rows, int64_t ldq_rows, float *s_rows,
                             int64_t ld_s_rows, int scale_mode, void *stream);

/*
 * 128x1 requantisation of FP8-cached activations: the forward pass keeps its
 * activations as 1x128-quantised E4M3 ([dssusan] paragraph 2: cached
 * activations are stored in low precision), and the backward pass needs the
 * same tensor in 128x1 tiles ([dssusan] paragraph 4).  Each cached value is
 * dequantised with one FP32 multiply, x = fl32(decode(q[t][c]) * s_rows(t, c)),
 * then quantised exactly as fp8q_quant_act_T quantises x.
 *   q       E4M3 [T][ldq], columns [0, C).          T % 128 == 0, C % 128 == 0,
 *           T <= 65535 * 128, C <= 2^31 - 1 (else FP8Q_ERR_SHAPE).
 *   s_rows  FP32 1x128 scales of q: s_rows[(c/128) * ld_s_rows + t], ld_s_rows >= T.
 *   qT      E4M3 [C][ldqT], qT[c][t];  sT FP32 sT[(t/128) * ld_sT + c].
 * Alignment: q, qT 16-byte aligned; ldq % 16 == 0, ldqT % 16 == 0.
 */
fp8q_status fp8q_requant_act_T(const void *q, int64_t T, int64_t C, int64_t ldq,
                               const float *s_rows, int64_t ld_s_rows, void *qT, int64_t ldqT,
                               float *sT, int64_t ld_sT, int scale_mode, void *stream);

/*
 * Weight quantisation, 128x128 blocks: one scale per 128 rows (output
 * channels) x 128 columns (input channels) ([dssusan] paragraph 4, Figure
 * 7 (a)(2)).  A last partial block of rows covers only the rows that exist.
 *   w   BF16 [N][ldw], columns [0, K).              K % 128 == 0, N >= 0.
 *   q   E4M3 [N][ldq].
 *   qT  optional (NULL to skip): E4M3 [K][ldqT], qT[k][n] = q[n][k] -- the
 *       K-major B operand of the Dgrad GEMM (dX = dY * W).
 *   sb  FP32 [ceil(N/128)][ld_sb], block (nb, kb) at sb[nb * ld_sb + kb],
 *       ld_sb >= K/128.
 * Alignment: w, q, qT 16-byte aligned; ldw % 8, ldq % 16, ldqT % 16 == 0.
 */
fp8q_status fp8q_quant_weight(const void *w, int64_t N, int64_t K, int64_t ldw,
                              void *q, int64_t ldq, void *qT, int64_t ldqT,
                              float *sb, int64_t ld_sb, int scale_mode,
                              void *stream);

/*
 * Per-tensor quantisation, for comparison with the fine-grained quantisers:
 * one scale for the whole tensor from its max-abs value, by the same rule as
 * a group's.  This is the standard practice the pages contrast with the
 * method ("Deepseek - Not For everyone", paragraph 4: mapping the tensor's
 * max-abs onto the FP8 maximum makes the result sensitive to outliers).
 * Two passes: per-64-row partial max-abs values go to `workspace`, then every
 * slab reduces them and quantises.
 *   x  BF16 [M][ldx], columns [0, K), K % 8 == 0;  q E4M3 [M][ldq];
 *   s  one FP32 (device) -- the tensor's scale.
 *   workspace  device scratch of at least fp8q_quant_tensor_workspace_bytes(M, K)
 *              bytes, 4-byte aligned, owned by the caller; its contents on entry
 *              do not matter.
 * Alignment: x, q 16-byte aligned; ldx % 8, ldq % 8 == 0.
 */
int64_t fp8q_quant_tensor_workspace_bytes(int64_t M, int64_t K);
fp8q_status fp8q_quant_tensor(const void *x, int64_t M, int64_t K, int64_t ldx,
                              void *q, int64_t ldq, float *s, void *workspace,
                              int64_t workspace_bytes, int scale_mode, void *stream);

/*
 * fp8q_quant_tensor with no workspace argument and no allocation.  The
 * sources describe no such call: it is a library convenience for callers that
 * cannot allocate device memory when they quantise (code inside an
 * allocator's or pool's callbacks, or a runtime whose device memory is all
 * handed to its own pools).  The scratch is a fixed 4 KB array in the
 * library's static device memory, one per device, so:
 *   - M <= 65536 (1024 partials of 64 rows); larger M returns FP8Q_ERR_SHAPE
 *     and launches nothing.  Every other argument, result and error is as for
 *     fp8q_quant_tensor.
 *   - The first call on a device (with that device current) looks up the
 *     array's device address; make that call before any stream capture.  The
 *     address is remembered with the id of the CUDA context it belongs to and
 *     looked up again when another context is current, e.g. after
 *     cudaDeviceReset or after the primary context was released and created
 *     again (the first call after that is again a set-up call).
 *   - Every call on a device uses the same array.  Calls whose kernels
 *     overlap on the GPU (different streams, no ordering between them) race
 *     and may return wrong scales; calls ordered on one stream do not.
 * The call makes no cudaMalloc or cudaFree and allocates no other memory.
 */
fp8q_status fp8q_quant_tensor_noalloc(const void *x, int64_t M, int64_t K, int64_t ldx,
                                      void *q, int64_t ldq, float *s, int scale_mode,
                                      void *stream);

/*
 * FP8 GEMM with per-group scaling along K ([dssusan] paragraph 3, Figure 6;
 * [youlimart] paragraph 2):
 *   C[m][n] = sum over 128-wide groups kb of
 *             sa(m,kb) * sb(n,kb) * sum_{k in kb} decode(a[m][k]) * decode(b[n][k])
 * The inner sums run on the tensor cores into an FP32 partial per group; each
 * partial is scaled and added into an FP32 accumulator by separate warps.
 * The result is stored as FP32, or rounded to nearest-even BF16.
 *   a   E4M3 [M][lda] (K-major), sa FP32 at sa[kb * ld_sa + m], ld_sa >= M.
 *   b   E4M3 [N][ldb] (K-major), sb FP32 laid out per bscale_kind (see enum).
 *   c   [M][ldc] BF16 or FP32 per out_dtype.
 *   K % 128 == 0; M, N >= 0 (tails are masked).  K == 0 writes zeros.
 * Alignment: a, b, c 16-byte aligned; lda % 16 == 0, ldb % 16 == 0,
 * ldc * sizeof(out) % 16 == 0.
 * Fprop: a = quantised activations, b = quantised weight, BLOCK scales.
 * Dgrad: a = quantised dY, b = the weight's qT, BLOCK_T over the weight's sb.
 * Wgrad: a = dY's qT, b = X's qT, sa = dY's sT, sb = X's sT with ROW scales.
 */
fp8q_status fp8q_gemm(const void *a, int64_t lda, const float *sa,
                      int64_t ld_sa, const void *b, int64_t ldb,
                      const float *sb, int64_t ld_sb, int bscale_kind, void *c,
                      int64_t ldc, int out_dtype, int64_t M, int64_t N,
                      int64_t K, void *stream);

/*
 * Gradient accumulation form of fp8q_gemm: C += the same product, C FP32.
 * Weight gradients are kept in FP32 and summed over micro-batches
 * ([dssusan] paragraph 2: weight gradients stay in FP32); each element
 * receives one FP32 addition, fl32(C_old + result).  Arguments and rules as
 * fp8q_gemm with out_dtype = FP8Q_OUT_FP32.
 */
fp8q_status fp8q_gemm_accumulate(const void *a, int64_t lda, const float *sa,
                                 int64_t ld_sa, const void *b, int64_t ldb,
                                 const float *sb, int64_t ld_sb, int bscale_kind,
                                 float *c, int64_t ldc, int64_t M, int64_t N,
                                 int64_t K, void *stream);

/*
 * fp8q_gemm for power-of-two scales, on the tensor cores' block-scaled MMA.
 * The method allows scaling factors that are integral powers of two
 * ([dssusan] paragraph 1) and recommends tensor cores that take the group
 * scales themselves ([dssusan] paragraph 3); Blackwell's microscaling MMA
 * ("Deepseek - Not For everyone", paragraph 3) multiplies each 32-wide K
 * block of A and B by a power of two inside the MMA.  This call computes the
 * same product as fp8q_gemm, with the K-group scales applied by the MMA and
 * the sum over all K-groups accumulated in FP32 by the tensor cores (no
 * per-group FP32 fold by the CUDA cores).
 *   Arguments, layouts, alignment and return codes: as fp8q_gemm.
 *   Precondition: every scale the product reads (sa of rows < M, sb of
 *   columns < N, K-groups < K/128) is a power of two 2^e, -127 <= e <= 127 --
 *   what the quantisers produce with FP8Q_SCALE_POW2.  Any other value is
 *   used by its binary exponent alone, and the kernel records
 *   FP8Q_ERR_INVALID in a device status word that fp8q_sync_status reports.
 *   K == 0 writes zeros (fp8q_gemm_pow2) or leaves C unchanged (_accumulate).
 * Tiles are 256 x 256 (a pair of CTAs per tile).
 */
fp8q_status fp8q_gemm_pow2(const void *a, int64_t lda, const float *sa,
                           int64_t ld_sa, const void *b, int64_t ldb,
                           const float *sb, int64_t ld_sb, int bscale_kind,
                           void *c, int64_t ldc, int out_dtype, int64_t M,
                           int64_t N, int64_t K, void *stream);

/* C (FP32) += the fp8q_gemm_pow2 product; as fp8q_gemm_accumulate otherwise. */
fp8q_status fp8q_gemm_pow2_accumulate(const void *a, int64_t lda, const float *sa,
                                      int64_t ld_sa, const void *b, int64_t ldb,
                                      const float *sb, int64_t ld_sb, int bscale_kind,
                                      float *c, int64_t ldc, int64_t M, int64_t N,
                                      int64_t K, void *stream);

/*
 * Grouped FP8 GEMM for MoE experts: rows [offs[g], offs[g+1]) of A (tokens
 * sorted by expert, top-1 routing) are multiplied by expert g's weight.
 *   a     E4M3 [M][lda], sa at sa[kb * ld_sa + m] as in fp8q_gemm.
 *   b     E4M3 [G][N][ldb] (expert g's rows start at b + g*N*ldb).
 *   sb    FP32 [G][ceil(N/128)][K/128] (BLOCK layout per expert).
 *   offs  int32 DEVICE array [G+1]: 0 <= offs[0] <= ... <= offs[G] <= M.
 *         Empty experts are allowed.  Rows outside [offs[0], offs[G]) are
 *         not written.  Offsets that break the ordering are clamped into
 *         [0, M] and a decreasing step is treated as an empty expert.
 *   c     [M][ldc] BF16 or FP32.
 *   1 <= G <= 1024; other rules as fp8q_gemm.
 */
fp8q_status fp8q_grouped_gemm(const void *a, int64_t lda, const float *sa,
                              int64_t ld_sa, const void *b, int64_t ldb,
                              const float *sb, const int32_t *offs, int G,
                              void *c, int64_t ldc, int out_dtype, int64_t M,
                              int64_t N, int64_t K, void *stream);

/*
 * fp8q_grouped_gemm for power-of-two scales, on the block-scaled MMA (see
 * fp8q_gemm_pow2): the same arguments, layouts and results, with the same
 * precondition on the scales.  Tiles are 256 rows x 256 columns (a CTA pair);
 * K must be a positive multiple of 128 (K == 0 returns FP8Q_ERR_SHAPE).
 */
fp8q_status fp8q_grouped_gemm_pow2(const void *a, int64_t lda, const float *sa,
                                   int64_t ld_sa, const void *b, int64_t ldb,
                                   const float *sb, const int32_t *offs, int G,
                                   void *c, int64_t ldc, int out_dtype, int64_t M,
                                   int64_t N, int64_t K, void *stream);

/*
 * Gated feed-forward block (SwiGLU), both projections, the activation and the
 * product in one kernel, from FP8 operands as fp8q_gemm takes them:
 *   g = X Wg^T, u = X Wu^T (per-128-K-group scales, FP32 sums),
 *   h = silu(g) * u,  silu(g) = g / (1 + exp(-g)), in FP32.
 *   a   E4M3 [M][lda] codes of X, sa FP32 at sa[kb * ld_sa + m].
 *   b   E4M3 [2F][ldb]: Wg in rows [0, F), Wu in rows [F, 2F), one matrix as
 *       fp8q_quant_weight quantises it; sb FP32 [2F/128][ld_sb] (BLOCK layout).
 * Results, each optional (NULL to skip), at least one required:
 *   h   BF16 [M][ldh], rounded to nearest-even.
 *   gu  BF16 [M][ld_gu]: g in columns [0, F), u in [F, 2F) -- what the
 *       backward pass (fp8q_swiglu_bwd) reads.
 *   q   E4M3 [M][ldq] with s FP32 at s[(f/128) * ld_s + m]: the 1x128
 *       quantisation, by scale_mode, of the unrounded FP32 h -- the A operand
 *       of the down projection's fp8q_gemm.
 * M >= 0; F % 128 == 0, K % 128 == 0; K == 0 gives g = u = h = 0.
 * Alignment: a, b, h, gu, q 16-byte aligned; lda, ldb, ldq % 16, ldh, ld_gu
 * % 8 == 0.  The inputs' scales may come from either scale mode.
 */
fp8q_status fp8q_gemm_swiglu(const void *a, int64_t lda, const float *sa, int64_t ld_sa,
                             const void *b, int64_t ldb, const float *sb, int64_t ld_sb,
                             void *h, int64_t ldh, void *gu, int64_t ld_gu, void *q,
                             int64_t ldq, float *s, int64_t ld_s, int scale_mode, int64_t M,
                             int64_t F, int64_t K, void *stream);

/*
 * fp8q_gemm_swiglu for power-of-two input scales, on the block-scaled MMA: the
 * same arguments and results, with fp8q_gemm_pow2's precondition on sa and sb.
 */
fp8q_status fp8q_gemm_swiglu_pow2(const void *a, int64_t lda, const float *sa, int64_t ld_sa,
                                  const void *b, int64_t ldb, const float *sb, int64_t ld_sb,
                                  void *h, int64_t ldh, void *gu, int64_t ld_gu, void *q,
                                  int64_t ldq, float *s, int64_t ld_s, int scale_mode,
                                  int64_t M, int64_t F, int64_t K, void *stream);

/*
 * fp8q_gemm_swiglu for MoE experts: rows [offs[g], offs[g+1]) of A meet expert
 * g's two projections.
 *   b     E4M3 [G][2F][ldb], sb FP32 [G][2F/128][K/128].
 *   offs  int32 DEVICE array [G+1], as for fp8q_grouped_gemm: rows outside
 *         [offs[0], offs[G]) are not written, in any of the results.
 *   1 <= G <= 1024; other rules as fp8q_gemm_swiglu.
 */
fp8q_status fp8q_grouped_gemm_swiglu(const void *a, int64_t lda, const float *sa, int64_t ld_sa,
                                     const void *b, int64_t ldb, const float *sb,
                                     const int32_t *offs, int G, void *h, int64_t ldh, void *gu,
                                     int64_t ld_gu, void *q, int64_t ldq, float *s, int64_t ld_s,
                                     int scale_mode, int64_t M, int64_t F, int64_t K,
                                     void *stream);

/* fp8q_grouped_gemm_swiglu for power-of-two input scales (block-scaled MMA). */
fp8q_status fp8q_grouped_gemm_swiglu_pow2(const void *a, int64_t lda, const float *sa,
                                          int64_t ld_sa, const void *b, int64_t ldb,
                                          const float *sb, const int32_t *offs, int G, void *h,
                                          int64_t ldh, void *gu, int64_t ld_gu, void *q,
                                          int64_t ldq, float *s, int64_t ld_s, int scale_mode,
                                          int64_t M, int64_t F, int64_t K, void *stream);

/*
 * Backward pass of the gated product, down to the gradients d = [dg | du] of
 * the two projections' outputs, in one pass over dh and the forward's gu:
 *   du = dh * silu(g),  dg = dh * u * s * (1 + g * (1 - s)),  s = 1/(1+exp(-g)).
 *   dh  BF16 [T][ld_dh], columns [0, F);  gu BF16 [T][ld_gu], columns [0, 2F).
 * Results, each optional (NULL to skip), at least one required:
 *   d   BF16 [T][ld_d], dg in columns [0, F), du in [F, 2F).
 *   q   E4M3 [T][ldq], columns [0, 2F), s FP32 at s[(c/128) * ld_s + t]: the
 *       1x128 quantisation of the unrounded FP32 d -- the A operand of
 *       dX = d [Wg; Wu] (fp8q_gemm over K = 2F with the weight's qT, BLOCK_T).
 *   qT  E4M3 [2F][ldqT], sT FP32 at sT[(t/128) * ld_sT + c]: the 128x1
 *       quantisation of d, transposed -- the A operand of the two projections'
 *       Wgrad.  T % 128 == 0.
 *   hT  E4M3 [F][ld_hT], shT FP32 at shT[(t/128) * ld_shT + c]: the 128x1
 *       quantisation of h = silu(g) * u (recomputed from gu, unrounded),
 *       transposed -- the B operand of the down projection's Wgrad.
 *       T % 128 == 0.
 * F % 128 == 0, T <= 65535 * 128.  Alignment: all tensors 16-byte aligned;
 * ld_dh, ld_gu, ld_d % 8, ldq, ldqT, ld_hT % 16 == 0.
 */
fp8q_status fp8q_swiglu_bwd(const void *dh, int64_t ld_dh, const void *gu, int64_t ld_gu,
                            void *d, int64_t ld_d, void *q, int64_t ldq, float *s, int64_t ld_s,
                            void *qT, int64_t ldqT, float *sT, int64_t ld_sT, void *hT,
                            int64_t ld_hT, float *shT, int64_t ld_shT, int64_t T, int64_t F,
                            int scale_mode, void *stream);

/*
 * Orthogonalised update of a weight gradient by Newton-Schulz steps, for a
 * batch of matrices (gradients leave fp8q_gemm_accumulate as FP32 [m][n]):
 *   X = G / (|G|_F + eps), oriented with the shorter side as its rows;
 *   steps times:  A = X X^T,  B = b A + c A^2,  X = a X + B X;
 *   out = X in G's orientation.
 * Products take FP16 operands (X, A, B scaled by 2^8) with FP32 sums.
 *   g    FP32 or BF16 (in_dtype: FP8Q_OUT_FP32 / FP8Q_OUT_BF16) [m][ldg],
 *        matrix i at g + i * g_stride elements.
 *   out  FP32 or BF16 (out_dtype) [m][ldo], matrix i at out + i * o_stride;
 *        may not overlap g or the workspace.
 *   1 <= steps <= 1000, eps >= 0 (a zero matrix with eps > 0 gives zeros).
 *   Limits: 0 <= m, n <= 2^20, batch <= 65535, and fewer than 2^30 units of
 *   work (256 x 64 tiles of the update's product times 64-wide blocks of its
 *   inner dimension: a 65536 x 65536 matrix passes); the sum of G's squares
 *   must be an FP32 value, and |a|, |b|, |c| such that the entries of X, A and B stay
 *   below 255 (FP16 after scaling; the usual coefficients keep them below 12).
 *   workspace  device scratch of at least
 *              fp8q_newton_schulz_workspace_bytes(batch, m, n) bytes, 256-byte
 *              aligned, owned by the caller; contents on entry do not matter.
 * g and out need only their element's alignment, at any pitch >= n.
 * workspace_bytes returns 0 for sizes outside the limits.
 */
int64_t fp8q_newton_schulz_workspace_bytes(int64_t batch, int64_t m, int64_t n);
fp8q_status fp8q_newton_schulz(const void *g, int64_t ldg, int64_t g_stride, int in_dtype,
                               void *out, int64_t ldo, int64_t o_stride, int out_dtype,
                               int64_t batch, int64_t m, int64_t n, int steps, float a, float b,
                               float c, float eps, void *workspace, int64_t workspace_bytes,
                               void *stream);

/*
 * Root-mean-square norm with the residual's addition, and the FP8 operand of
 * the product behind it, in one pass over each row:
 *   h = x + res,  rstd = 1 / sqrt(sum(h^2) / C + eps),  y = h * rstd * w, in FP32.
 *   x     [T][ldx] and res (optional, NULL: h = x) [T][ld_res], BF16 or FP32 each
 *         (x_dtype, res_dtype: FP8Q_OUT_BF16 / FP8Q_OUT_FP32); w [C] BF16 or FP32.
 * Results, each optional (NULL to skip), at least one required:
 *   r     [T][ld_r] of res_dtype: h, the new residual stream, rounded to
 *         nearest-even (needs res; may be res itself, with its pitch).
 *   y     BF16 [T][ldy].
 *   q     E4M3 [T][ldq] with s FP32 at s[(c/128) * ld_s + t]: the 1x128
 *         quantisation, by scale_mode, of the unrounded FP32 y -- the A operand
 *         of fp8q_gemm and of fp8q_gemm_swiglu.  C % 128 == 0.
 *   rstd  FP32 [T], what fp8q_rmsnorm_bwd reads.  Not with C == 0.
 * The norm is of the unrounded h.  A row of zeros with eps > 0 gives zeros.
 * T >= 0, 0 <= C <= 32768, C % 8 == 0, eps >= 0; a row's sum of squares must be
 * an FP32 value.  Alignment: x, res, w, r, y, q 16-byte aligned; every pitch a
 * multiple of 16 bytes.
 */
fp8q_status fp8q_rmsnorm(const void *x, int64_t ldx, int x_dtype, const void *res, int64_t ld_res,
                         int res_dtype, const void *w, int w_dtype, float eps, void *r,
                         int64_t ld_r, void *y, int64_t ldy, void *q, int64_t ldq, float *s,
                         int64_t ld_s, float *rstd, int scale_mode, int64_t T, int64_t C,
                         void *stream);

/*
 * Backward pass of fp8q_rmsnorm: with xh = x * rstd and c the row's mean of
 * dy * w * xh,
 *   dx = rstd * (dy * w - xh * c) + dres,   dw = sum over rows of dy * xh.
 *   dy    [T][ld_dy] BF16 or FP32; x [T][ldx] BF16 or FP32: the normalised rows
 *         (the forward's r, or its x where there was no residual);
 *         rstd FP32 [T]; w [C] BF16 or FP32.
 *   dres  optional (NULL: 0) [T][ld_dres] of out_dtype: the gradient that
 *         reaches r on the residual stream itself.  May be dx itself.
 * Results, at least one required:
 *   dx    [T][ld_dx] of out_dtype: the gradient of x and of res alike.
 *   dw    FP32 [C]; added to what it holds where accumulate is not 0.  Summed in
 *         an order that depends on T, C and the types alone.  T == 0 gives zeros.
 *   workspace  for dw: device scratch of fp8q_rmsnorm_bwd_workspace_bytes(T, C)
 *              bytes (0 for sizes outside the limits), 16-byte aligned, owned by
 *              the caller; contents on entry do not matter.
 * Limits and alignment as for fp8q_rmsnorm.
 */
int64_t fp8q_rmsnorm_bwd_workspace_bytes(int64_t T, int64_t C);
fp8q_status fp8q_rmsnorm_bwd(const void *dy, int64_t ld_dy, int dy_dtype, const void *x,
                             int64_t ldx, int x_dtype, const float *rstd, const void *w,
                             int w_dtype, const void *dres, int64_t ld_dres, void *dx,
                             int64_t ld_dx, int out_dtype, float *dw, int accumulate, int64_t T,
                             int64_t C, void *workspace, int64_t workspace_bytes, void *stream);

/*
 * One AdamW step over a list of tensors:
 *   g' = g * grad_scale,  m = beta1 m + (1 - beta1) g',  v = beta2 v + (1 - beta2) g'^2,
 *   p = p - lr * (weight_decay p + (m / (1 - beta1^step)) /
 *                                  (sqrt(v / (1 - beta2^step)) + eps)), in FP32.
 * All tensors of a call have the same types:
 *   p     FP32 or BF16 (p_dtype), g FP32 or BF16 (g_dtype); BF16 values are
 *         rounded to nearest-even.
 *   copy  optional: BF16 [n], the new p rounded (what fp8q_quant_weight reads).
 *   m, v  by state_kind: FP32, BF16 (rounded to nearest-even; the step takes
 *         the unrounded values), or FP8Q_STATE_E4M3: m and sqrt(v) as E4M3 codes
 *         with one FP32 scale per 128 consecutive values (the last group may be
 *         shorter) in m_scale and v_scale: with a = max(amax, 2^-116) of the
 *         group, scale = a * (1 / 448) and codes E4M3(x * (448 * (1 / a))), each
 *         operation rounded to nearest; a positive sqrt(v) at least to the
 *         smallest code, 2^-9, so that no denominator becomes 0 by rounding.
 *         Zero bytes and scales are the state before the first step.
 * Moments of fewer than 32 bits are rounded after every step, and a step that
 * moves one by less than half of its last place leaves it where it is:
 *   BF16    v follows its gradients to within 2^-8 / (1 - beta2) of itself: 8 %
 *           at beta2 = 0.95, not at all at 0.999.
 *   8 bits  half a code step is 2^-5 to 2^-4 of m or sqrt(v).  With beta2 up to
 *           0.95 the changes of a group's largest value carry its codes along
 *           (normal gradients: a mean root of 1.06 times the exact one); with
 *           0.99 and more a value whose gradients shrink against its group's
 *           keeps its code, and its steps stay too small.
 * FP32 moments take any beta2.
 * A gradient that is no finite number makes its parameter NaN and leaves the
 * others alone; with moments in 8 bits an infinite one takes its group with it.
 * `tensors` is a HOST array, copied by the call.  Tensors are dense; none may
 * overlap another (the p, m, v of a call are checked, FP8Q_ERR_INVALID).
 *   lr, step   by value, or from device memory where lr_dev / step_dev are not
 *              NULL (a captured call then follows them); step counts from 1.
 *   grad_scale optional (NULL: 1) FP32 in device memory, e.g. a clipping factor.
 *   0 <= beta1, beta2 < 1, eps >= 0 (a positive one below 2^-126 counts as that; with
 *   0 a value whose gradients were all 0 becomes NaN); eps, lr, weight_decay at most
 *   the largest FP32 value; n >= 0, the tensors of a call below 2^42 values together.
 * Alignment: every address at its element's; tensors whose addresses are all
 * 16-byte aligned take wide loads.
 */
enum { FP8Q_STATE_BF16 = 0, FP8Q_STATE_FP32 = 1, FP8Q_STATE_E4M3 = 2 };
typedef struct fp8q_adamw_tensor {
  void *p;
  const void *g;
  void *m, *v;
  float *m_scale, *v_scale; /* FP8Q_STATE_E4M3 only */
  void *copy;               /* NULL: none */
  int64_t n;
} fp8q_adamw_tensor;
fp8q_status fp8q_adamw(const fp8q_adamw_tensor *tensors, int64_t count, int p_dtype, int g_dtype,
                       int state_kind, double lr, double beta1, double beta2, double eps,
                       double weight_decay, int64_t step, const float *lr_dev,
                       const int64_t *step_dev, const float *grad_scale, void *stream);

/*
 * Router of a mixture of experts: the choice of k experts for each token, the
 * weights of their sum, and the sorted order that the grouped products take.
 *   logits [T][ld] BF16 or FP32, columns [0, E).  An expert at -inf (or NaN) is
 *          closed to the token; +inf counts as the largest FP32 value.
 *   valid  optional (NULL: all) one byte per token, 0: a padding token, which
 *          goes to no expert and does not count.
 *   score  s_e = softmax(logits)_e over the open experts or sigmoid(logit_e).
 * Results, all required:
 *   idx    int32 [T][k]: the k largest logits in falling order, equal ones in
 *          rising order of e; -1 where no open expert is left.
 *   weight FP32 [T][k]: s of the choice, divided by the token's sum of them where
 *          normalise is not 0, times scale; 0 where idx is -1.
 *   counts int32 [E]: choices per expert.  offs int32 [E+1]: their exclusive sums,
 *          the offsets of fp8q_grouped_gemm.
 *   order  int32 [T*k]: choice t * k + j at each row of the order sorted by
 *          expert, within an expert by rising t; -1 behind row offs[E].
 *   slot   int32 [T][k]: each choice's row in that order, -1 where idx is -1.
 *   tokens int32 [1]: tokens with a choice.
 *   loss   FP32 [1]: the balance loss, E * sum_e f_e P_e with f_e expert e's share
 *          of all choices and P_e the mean over those tokens of s_e / sum s; 1
 *          where all experts are used alike, 0 without tokens.
 * Sums of scores below 2^-126 count as 2^-126.  With u = 2^-24, weights of sigmoid scores
 * are right to 18 u whatever the logit, of softmax scores to 70 u and the rounding of
 * logit - maximum; the probabilities s / sum s of the loss, and their gradient, to 70 u
 * and 4 |logit| u (sigmoid) or 2 |logit - maximum| u (softmax).
 *   1 <= k <= min(E, 32), E <= 1024, 0 <= T <= 2^26, T * k < 2^31.
 *   workspace  device scratch of fp8q_route_workspace_bytes(T, E) bytes (0 for
 *              sizes outside the limits), 16-byte aligned, owned by the caller;
 *              contents on entry do not matter.
 * idx, weight, order and slot are dense.  Alignment: every address at its
 * element's.  The same bits in every run.
 */
enum { FP8Q_SCORE_SOFTMAX = 0, FP8Q_SCORE_SIGMOID = 1 };
int64_t fp8q_route_workspace_bytes(int64_t T, int64_t E);
fp8q_status fp8q_route(const void *logits, int64_t ld, int dtype, const uint8_t *valid, int score,
                       int normalise, float scale, int32_t *idx, float *weight, int32_t *counts,
                       int32_t *offs, int32_t *order, int32_t *slot, int32_t *tokens, float *loss,
                       int64_t T, int64_t E, int64_t k, void *workspace, int64_t workspace_bytes,
                       void *stream);

/*
 * Backward pass of fp8q_route: the gradient of the logits from those of the
 * weights and of the balance loss.  The choice and the counts are constants.
 *   logits, valid, score, normalise, scale  as the forward call took them;
 *   idx, counts, tokens  its results.
 *   dweight  optional (NULL: 0) FP32 [T][k];  dloss optional (NULL: 0) FP32 [1].
 *   dlogits  [T][ld_d] of the logits' type: 0 at closed experts and padding.
 * An idx outside [0, E), of a closed expert or of a padding token is no choice: its
 * dweight does not count, whatever it holds (NaN, memory never written).
 */
fp8q_status fp8q_route_bwd(const void *logits, int64_t ld, int dtype, const uint8_t *valid,
                           int score, int normalise, float scale, const int32_t *idx,
                           const int32_t *counts, const int32_t *tokens, const float *dweight,
                           const float *dloss, void *dlogits, int64_t ld_d, int64_t T, int64_t E,
                           int64_t k, void *stream);

/*
 * Plain FP32 -> E4M3 conversion of n values (round to nearest-even, saturate
 * to +-448, NaN -> 0x7F), with no scaling.  The quantisers use the same
 * conversion; this entry exposes it so it can be checked on every FP32 bit
 * pattern.  x: FP32 [n], q: E4M3 [n]; both 16-byte aligned.
 */
fp8q_status fp8q_cast_e4m3(const float *x, int64_t n, void *q, void *stream);

/*
 * Synchronise `stream`, then read and clear this device's status words (one
 * small kernel and one copy on `stream`, which must not be capturing).
 * Returns FP8Q_ERR_TIMEOUT if a kernel's bounded wait gave up since the last
 * call, FP8Q_ERR_INVALID if a power-of-two call met another scale,
 * FP8Q_ERR_CUDA if synchronisation failed, else FP8Q_OK.
 */
fp8q_status fp8q_sync_status(void *stream);

/*
 * Set the time limit, in nanoseconds, of every device-side wait launched
 * afterwards from this process (default 2e9 = 2 s; 0 restores the default).
 */
void fp8q_set_wait_timeout_ns(uint64_t ns);

/*
 * Diagnostic: launch one CTA that waits, with the bounded wait the GEMM uses,
 * on a barrier that nothing ever completes, for at most timeout_ns.  The wait
 * must give up, record FP8Q_ERR_TIMEOUT in the status word and return; the
 * caller then reads it with fp8q_sync_status().
 */
fp8q_status fp8q_selftest_wait_timeout(uint64_t timeout_ns, void *stream);

/* Human-readable name of a status code (static storage). */
const char *fp8q_status_string(fp8q_status s);

/* ABI version of this header (major * 100 + minor). */
int fp8q_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FP8Q_H */
