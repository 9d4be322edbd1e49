/*
 * fp8bq -- operators of a decode step around the block-FP8 linear layer
 * (libfp8bq.so, gfx950): the norm in front of it with its 8-bit output, the
 * same layer in 8-bit integers, and the verification of drafted tokens behind
 * the vocabulary projection.
 *
 * Where they come from: page 3 (zskr.cn blog), section 3.3, fuses the
 * root-mean-square norm with the quantisation that follows it and section 2.2
 * stores weights as INT8; page 1 (SmartX blog), section "single-stream
 * optimisation", verifies k drafted tokens per step (M = k + 1 rows).
 *
 * The conventions of fp8bq.h hold for every call here: device pointers on the
 * current device, dense row-major tensors, buffers owned by the caller,
 * enqueued on `stream` without synchronising (and without allocating, so
 * every call may be captured into a HIP graph), arguments checked on the host
 * before anything is enqueued, FP8BQ_OK or a negative fp8bq_status returned.
 */
#ifndef FP8BQ_STEP_H
#define FP8BQ_STEP_H

#include <stdint.h>

#include "fp8bq.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Residual addition, root-mean-square norm and 8-bit output in one launch.
 *
 *   h   = bf16(x + r)                      (h = x without a residual)
 *   inv = fp32(1 / sqrt(mean_k(h^2) + eps)) (mean and root in 64 bits; held
 *                                          to the largest finite fp32 number)
 *   y   = bf16((h * inv) * weight)         (fp32 products)
 *   fp8bq_rmsnorm_quant:    codes, scales = fp8bq_quant_act(y)
 *   fp8bq_rmsnorm_quant_i8: codes, scales = fp8bq_quant_act_i8(y)
 *
 *   X_bf16  [M, K] bf16, read.
 *   R_bf16  [M, K] bf16, read: the residual stream; NULL for none.
 *   weight  [K] bf16, read.
 *   H_bf16  [M, K] bf16, written: the new residual stream h. Required with a
 *           residual (it may be R_bf16 or X_bf16 itself: each element is
 *           read before it is written), NULL or ignored without one.
 *   codes, scales: written, as fp8bq_quant_act / fp8bq_quant_act_i8 write
 *           them, which give the same bits for the same y. The mean square is
 *           summed in 64 bits, so the order of the sum shows in no code but
 *           where the root's inverse lies within about 2^-50 of the border
 *           between two fp32 numbers (one row in 10^7 or fewer).
 * M == 0 or K == 0 is a quick return that writes nothing (the scales of int8
 * rows without columns among it). NaN or infinite inputs give unspecified
 * codes in their row. Errors: NULL pointer; M < 0, K < 0, K % 128 != 0,
 * K > FP8BQ_NORM_MAX_K, M >= 2^31 or M*K > 2^40; eps not finite or <= 0
 * (FP8BQ_ERR_VALUE); X_bf16, R_bf16, weight, H_bf16 or codes not 16-B
 * aligned, scales not 4-B aligned; device not gfx950.
 */
#define FP8BQ_NORM_MAX_K 65536
int fp8bq_rmsnorm_quant(int64_t M, int64_t K, const void *X_bf16, const void *R_bf16, const void *weight,
                        double eps, void *H_bf16, void *A_fp8, float *A_scales, void *stream);
int fp8bq_rmsnorm_quant_i8(int64_t M, int64_t K, const void *X_bf16, const void *R_bf16, const void *weight,
                           double eps, void *H_bf16, void *A_i8, float *A_scales, void *stream);

/*
 * Quantisation to 8-bit integers, one scale per row.
 *
 *   scale = amax / 127 (IEEE fp32 division, amax over the row; 1.0 where it
 *   is 0: an all-zero row, or an amax below 2^-143),
 *   code = rint(x / scale) (ties to even), held to -127 .. 127.
 *
 * fp8bq_quant_act_i8:    A_bf16 [M, K] bf16 -> A_i8 [M, K] int8, A_scales [M]
 *                        fp32: one scale per token.
 * fp8bq_quant_weight_i8: W_f32 [N, K] fp32 -> W_i8 [N, K] int8, W_scales [N]
 *                        fp32: one scale per output channel.
 * Bit-exact with the definition for finite inputs. M == 0, N == 0 or K == 0
 * is a quick return that writes nothing. Errors: as fp8bq_quant_act, K > FP8BQ_NORM_MAX_K, and
 * M, N >= 2^31.
 */
int fp8bq_quant_act_i8(int64_t M, int64_t K, const void *A_bf16, void *A_i8, float *A_scales, void *stream);
int fp8bq_quant_weight_i8(int64_t N, int64_t K, const float *W_f32, void *W_i8, float *W_scales, void *stream);

/*
 * Matrix product in 8-bit integers with a scale per token and per channel.
 *
 *   C[m, n] = bf16( fp32( sum_k A_i8[m, k] * W_i8[n, k] )
 *                   * (A_scales[m] * W_scales[n]) )
 *
 *   A_i8 [M, K] int8, A_scales [M] fp32, W_i8 [N, K] int8, W_scales [N] fp32
 *   (read); C_bf16 [M, N] bf16 (written). Every code value serves, -128
 *   included. The sum is exact in 32-bit integers, so C does not depend on
 *   the kernel, the tile or the workspace that computed it; the sum is
 *   rounded to fp32, multiplied by the product of the two scales in fp32 and
 *   rounded to bf16 (RNE).
 *   workspace        device scratch, 16-B aligned, workspace_bytes long (NULL
 *                    only with workspace_bytes == 0), not overlapping the
 *                    other arguments; overwritten, contents on entry ignored.
 *                    Calls sharing a workspace must be ordered.
 *   workspace_bytes  >= fp8bq_gemm_i8_workspace_bytes(M, N, K): the K range
 *                    of each tile may be split over several workgroups;
 *                    below it (0 included) it is not. Same result.
 * M == 0 or N == 0 is a quick return; K == 0 writes zeros. Errors: NULL
 * pointer; negative size; K % 128 != 0; K > FP8BQ_GEMM_I8_MAX_K (sums then
 * leave 32 bits); M*K, N*K or M*N > 2^40; M or N >= 2^31; M > 64 with 2^23
 * or more tiles of 256 tokens x 256 weight rows; workspace_bytes < 0; codes, C_bf16 or workspace not 16-B aligned, scales not 4-B aligned;
 * device not gfx950.
 *
 * fp8bq_gemm_i8_workspace_bytes: the scratch the plan for (M, N, K) takes
 * (0: none), or a negative status for sizes fp8bq_gemm_i8 rejects. Host-only.
 */
#define FP8BQ_GEMM_I8_MAX_K 130944
int64_t fp8bq_gemm_i8_workspace_bytes(int64_t M, int64_t N, int64_t K);
int fp8bq_gemm_i8(int64_t M, int64_t N, int64_t K, const void *A_i8, const float *A_scales, const void *W_i8,
                  const float *W_scales, void *C_bf16, void *workspace, int64_t workspace_bytes, void *stream);

/*
 * Verification of drafted tokens against the target's probabilities, from
 * given random numbers.
 *
 * Draft i of sequence b, token d = drafts[b, i], is accepted iff
 *   u_accept[b, i] * q < p,  p = target_p[b, i, d], q = draft_p[b, i, d]
 * (exact products; q = 1 without draft_p, the drafts then being certain).
 * The first draft that is not accepted, at place r, ends the drafts (r =
 * their number where all are), and one more token is drawn from
 *   max(target_p[b, r, :] - draft_p[b, r, :], 0)   where draft r was rejected
 *   target_p[b, r, :]                              where none was
 * (without draft_p, 1 is subtracted at the rejected token alone). Where the
 * first has no weight at all, the second is drawn from.
 *
 * The draw. Weight w (fp32) counts as the whole number of 2^-32 nearest to it
 * (ties to even; below 0 and NaN as 0, at most 2^32 - 1); with S their sum
 * and z = floor(u_sample[b] * 2^32), the token is the lowest v whose sum of
 * weights 0 .. v exceeds floor(S z / 2^32). All of it is in whole numbers:
 * the result does not depend on the order of a sum. Weights below 2^-33 are
 * never drawn.
 *
 *   dtype     FP8BQ_F32 or FP8BQ_BF16: the type of both probability tensors.
 *   target_p  [B, drafts + 1, V], read (row r of each sequence, and single
 *             values). draft_p [B, drafts, V], read the same way; NULL: the
 *             drafts are certain.
 *   drafts    [B, n_drafts] int32, read; a token outside [0, V) is rejected.
 *   draft_len [B] int32, read: sequence b has the first draft_len[b] of its
 *             drafts (held to 0 .. n_drafts); NULL: all of them.
 *   u_accept  [B, n_drafts] fp32, u_sample [B] fp32, read: in [0, 1).
 *   workspace device scratch of workspace_bytes >=
 *             fp8bq_verify_workspace_bytes(B, n_drafts, V), 16-B aligned;
 *             contents on entry ignored. Calls sharing it must be ordered.
 *   tokens    [B, n_drafts + 1] int32, written: the accepted drafts, the
 *             drawn token, then -1. The drawn token is -1 where its row has
 *             no weight at all.
 *   accepted  [B] int32, written: r.
 * B == 0 is a quick return. Errors: n_drafts < 0 or > FP8BQ_MAX_DRAFTS;
 * V < 1 or V >= 2^31; B < 0 or B > 65535; B * (n_drafts + 1) * V > 2^40;
 * another dtype (FP8BQ_ERR_VALUE); workspace_bytes too small; NULL pointer
 * (drafts and u_accept may be NULL with n_drafts == 0); workspace not 16-B,
 * fp32 and int32 tensors not 4-B, bf16 tensors not 2-B aligned; device not
 * gfx950.
 */
#define FP8BQ_MAX_DRAFTS 64
enum { FP8BQ_F32 = 0, FP8BQ_BF16 = 1 };
int64_t fp8bq_verify_workspace_bytes(int64_t B, int64_t n_drafts, int64_t V);
int fp8bq_verify_drafts(int64_t B, int64_t n_drafts, int64_t V, int dtype, const void *target_p, const void *draft_p,
                        const int32_t *drafts, const int32_t *draft_len, const float *u_accept,
                        const float *u_sample, void *workspace, int64_t workspace_bytes, int32_t *tokens,
                        int32_t *accepted, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8BQ_STEP_H */
