/*
 * tn_experts.h -- expert layers in FP8: routing tokens to experts, putting the
 * (token, expert) pairs in expert order, quantising operands in blocks of 128, and
 * the TN products of such operands, plain and grouped by expert.
 *
 * The conventions of tn_gemm.h hold: device pointers owned by the caller, no call
 * allocates, arguments are checked on the host before anything is launched, calls are
 * asynchronous on `stream`, and pointers are 16-byte aligned except where a smaller
 * alignment is stated.  A call whose token or row count is 0 does nothing and returns
 * GEMM_OK (its pointers may then be NULL).  Outputs may not overlap inputs.
 */
#ifndef TN_EXPERTS_H
#define TN_EXPERTS_H

#include "tn_gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { GEMM_DT_F32 = 0, GEMM_DT_BF16 = 1, GEMM_DT_F16 = 2 }; /* element types          */
enum { ROUTE_SIGMOID = 0, ROUTE_SOFTMAX = 1 };               /* scoring of expert_route */

/*
 * Router.  For each token t, with x = logits[t][.]:
 *
 *   s_e   = 1 / (1 + exp(-x_e))  (ROUTE_SIGMOID)  or  softmax(x)_e  (ROUTE_SOFTMAX)
 *   key_e = s_e + bias[e], or, without a bias, x_e itself (the order of the scores,
 *           free of their rounding).  The bias takes part in the choice alone.
 *   groups > 1: the experts form `groups` runs of E / groups.  A run's score is the sum
 *           of its group_best (1 or 2) best s_e + bias[e] (without a bias: of its best
 *           s_e; of its best x_e where group_best is 1).  The top_groups best runs are
 *           kept, the lower run first among equals; the others' experts are not chosen.
 *   ids[t][.]     = the top_k experts with the largest keys, in descending order, the
 *                   lower index first among equal keys.
 *   weights[t][j] = scale * s_j / sum_i s_i over the chosen (renormalize != 0; 0 where
 *                   that sum is 0), or scale * s_j.  Renormalised shares of a softmax are
 *                   exp(x_j - max of the chosen x) over their sum, however far the chosen
 *                   lie below the row's largest.
 *
 * A logit of -inf masks its expert: it is chosen only when nothing else is left in the
 * kept runs, its weight is 0, and it adds nothing to its run's score (a run of masked
 * experts alone comes last).  NaN counts as -inf.  Scores and sums are fp32.
 *
 *   0 <= T < 2^31, 1 <= E <= 1024, 1 <= top_k <= 32, 1 <= groups <= 32 with E % groups == 0,
 *   top_k <= top_groups * E / groups.
 *   logits   [T] rows of E elements of `dtype` (GEMM_DT_*), ld elements apart
 *            (E <= ld < 2^31); aligned to its element.
 *   bias     float[E] or NULL.
 *   weights  float[T][top_k].       ids  int32[T][top_k].   (4-byte aligned)
 */
gemm_status_t expert_route(int64_t T, int64_t E, int64_t top_k, const void *logits, int64_t ld, int dtype,
                           const float *bias, float *weights, int32_t *ids, int scoring, int64_t groups,
                           int64_t top_groups, int group_best, int renormalize, float scale, cudaStream_t stream);

/*
 * Gradient of expert_route's weights with respect to the logits, the choice held fixed
 * (the bias has no gradient).  With g = dweights[t][.] and the chosen scores s_j, S their
 * sum:
 *   ds_j = scale * (g_j - sum_i g_i s_i / S) / S   (renormalize; 0 where S is 0)
 *   ds_j = scale * g_j                             (otherwise)
 *   ROUTE_SIGMOID  dlogits_e = ds_j s_j (1 - s_j) where e was chosen, else 0
 *   ROUTE_SOFTMAX  dlogits_e = s_e (ds_e - sum_j ds_j s_j), ds_e = 0 where not chosen
 * rounded once to `dtype`.  An id outside 0 .. E-1 stands for no expert and is skipped;
 * the ids of a token are distinct.
 *   dlogits  [T] rows of E elements of `dtype`, ldd elements apart (E <= ldd < 2^31; the
 *            elements between rows are not written).
 */
gemm_status_t expert_route_grad(int64_t T, int64_t E, int64_t top_k, const void *logits, int64_t ld, int dtype,
                                const int32_t *ids, const float *dweights, void *dlogits, int64_t ldd, int scoring,
                                int renormalize, float scale, cudaStream_t stream);

/*
 * The T * top_k pairs p = t * top_k + j in expert order (a stable counting sort):
 *   offsets[e]      pairs of experts below e; offsets[E] = pairs of all experts
 *   order[i]        the pair at place i; -1 from place offsets[E] on
 *   position[p]     the place of pair p; -1 for a pair whose id is outside 0 .. E-1
 *                   (a dropped pair)
 * Pairs of one expert keep their order, whatever the launch: results are deterministic.
 *   T >= 0, top_k >= 1, T * top_k < 2^31, 1 <= E <= 1024.
 *   ids int32[T * top_k], offsets int32[E + 1], order and position int32[T * top_k]
 *   (4-byte aligned).  With T == 0 offsets are still written (all 0).
 */
gemm_status_t expert_group(int64_t T, int64_t top_k, int64_t E, const int32_t *ids, int32_t *offsets, int32_t *order,
                           int32_t *position, cudaStream_t stream);

/*
 * FP8 E4M3 codes with one fp32 scale per block of 128 elements:
 *   a   = max(largest |x| of the block, 2^-100)
 *   SF  = a / 448,   Q = round_e4m3(x * (448 / a)), to nearest even,
 * each operation rounded to fp32: a code is the nearest of x / SF except where x / SF lies
 * within 2^-22 of its value from the middle of two codes, which may go either way.
 * (The lower bound on a keeps both factors finite; a block of zeros gets codes 0.)  A NaN
 * keeps its own code NaN and does not enter the block's maximum; a block with an
 * infinity gets an infinite scale and dequantises to NaN.
 *
 *   layout FP8_ROWS     blocks of 1 x 128 along a row: Q u8[R][K], SF float[R][ceil(K/128)];
 *                       K % 16 == 0.  With `index`, row i is X's row index[i] / index_div,
 *                       and a row of zeros where index[i] is negative or that row is not
 *                       below M; without, R must be M.
 *   layout FP8_COLS     blocks of 128 x 1 along a column, the output transposed:
 *                       Q u8[K][P], SF float[K][ceil(P/128)], P = M rounded up to a
 *                       multiple of 16; the codes past M are 0.  K % 8 == 0.
 *   layout FP8_TILES    blocks of 128 x 128: Q u8[M][K], SF float[ceil(M/128)][ceil(K/128)];
 *                       K % 16 == 0.
 *   layout FP8_TILES_T  the same blocks, codes and scales transposed:
 *                       Q u8[K][P], SF float[ceil(K/128)][ceil(P/128)].  K % 8 == 0.
 *
 *   M rows of X of K elements of `dtype`, ld elements apart (K <= ld < 2^31; ld * element size a
 *   multiple of 16).  R rows out (FP8_ROWS; else R is ignored).  `index` int32[R] or
 *   NULL; index_div >= 1.  SF and index 4-byte aligned.  1 <= K < 2^31 - 128;
 *   0 <= M, R < 2^31, and M <= 65535 * 128 in the layouts other than FP8_ROWS.
 */
enum { FP8_ROWS = 0, FP8_COLS = 1, FP8_TILES = 2, FP8_TILES_T = 3 };
gemm_status_t quantize_fp8(int64_t M, int64_t K, const void *X, int64_t ld, int dtype, int layout, int64_t R,
                           const int32_t *index, int64_t index_div, void *Q, float *SF, cudaStream_t stream);

/*
 * FP8 E4M3 TN GEMM with an fp32 scale per block of 128 along K:
 *   D[m][n] = round( C[m][n] + sum_b SFA[m][b] * SFB[.][b] * sum_{k in block b} A[m][k] * B[n][k] ).
 *   A u8[M][K] with SFA float[M][ceil(K/128)]; B u8[N][K] with
 *     scales FP8_ROWS   SFB float[N][ceil(K/128)]             (a scale per row and block)
 *     scales FP8_TILES  SFB float[ceil(N/128)][ceil(K/128)]   (a scale per 128 rows and block)
 *   C, D [M][N] of out_dtype (GEMM_DT_BF16 or GEMM_DT_F32); C may be NULL (0) or D itself.
 *   M >= 0; N, K >= 1; all < 2^31; K % 16 == 0, N % 8 == 0.  SFA, SFB 4-byte aligned.
 * The products of a block are summed in fp32 by the tensor cores; each block's sum is
 * scaled and added in fp32, C last, and the result is rounded once.  The order of the
 * additions depends on the sizes and the device alone.
 * Forward: FP8_TILES weights.  Gradient of the input: the same call on the weights'
 * FP8_TILES_T codes.  Gradient of the weights: FP8_ROWS scales on FP8_COLS codes of both
 * sides, added in fp32 (C == D).
 */
gemm_status_t gemm_fp8_block(int64_t M, int64_t N, int64_t K, const void *A, const float *SFA, const void *B,
                             const float *SFB, int scales, const void *C, void *D, int out_dtype, cudaStream_t stream);

/*
 * The same product for rows in expert order: rows offsets[e] .. offsets[e+1]-1 of A go
 * through B[e].  A u8[R][K], SFA float[R][ceil(K/128)], B u8[E][N][K],
 * SFB float[E][ceil(N/128)][ceil(K/128)], offsets int32[E+1] in device memory,
 * D bf16[R][N].  Rows outside every expert (from offsets[E] on) are not written; offsets
 * are read as if clamped to 0 .. R and made ascending.  1 <= E <= 1024; 0 <= R <= 2^31 - 512;
 * E * N <= 2^31 - 512; sizes and alignment otherwise as gemm_fp8_block.
 */
gemm_status_t gemm_fp8_block_grouped(int64_t R, int64_t N, int64_t K, int64_t E, const void *A, const float *SFA,
                                     const void *B, const float *SFB, const int32_t *offsets, void *D,
                                     cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* TN_EXPERTS_H */
