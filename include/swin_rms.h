/*
 * swin_block_rms -- the root-mean-square norm of the residual stream, with the
 * residual's addition in front of it, an output in bf16 or in 8 bits with
 * scales, and its backward pass, on one GB300 (sm_103a), behind a plain C ABI.
 *
 * Per token (row) of C channels, in fp32 from bf16 tensors:
 *   s = x + residual (rounded to bf16; s = x without a residual)
 *   r = 1 / sqrt(mean_c s^2 + eps)
 *   y = s r gamma
 * (fp32: a row whose squares add up to more than 3.4e38 has r = 0; with eps = 0,
 * one whose squares add up to less than 1.2e-38 has an inexact r, and a row of
 * zeros gives NaN, in the backward pass also in dgamma.)  The norm sees the
 * stored (rounded) sum, so that the backward pass, which starts from it,
 * differentiates the very function that ran.  8-bit output:
 * scale = max(max_c |y|, 1e-30) / 448 per row, code = y / scale (both fp32
 * quotients) rounded to nearest even in e4m3 (448 is its largest value), y ~
 * code * scale.  A row of zeros (eps > 0) gets zero codes and a positive scale;
 * a row holding an infinity or a NaN gets NaN codes and a NaN scale.
 *
 * Beside swin_stage_norm (LayerNorm): the other norm of the residual stream,
 * in front of swin_block_gated_forward (swin_gated.h), whose 8-bit form reads
 * the codes and scales written here.  Conventions of swin_wattn.h: device
 * pointers, asynchronous on `stream`, caller-owned tensors, status codes
 * SWIN_WATTN_*, no CPU fallback.
 */
#ifndef SWIN_RMS_H
#define SWIN_RMS_H

#include "swin_wattn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct swin_block_rms_s *swin_block_rms_t;

/* Rows of C channels (a multiple of 8, at most 16384) and eps >= 0 (finite).
 * *out receives the handle (NULL on failure).  EINVAL for bad arguments.  The
 * handle belongs to the device that is current at its first call that
 * launches; calls with another current device return EINVAL.  One handle may
 * be used on several streams (calls that need its workspace are ordered by an
 * event) but not from two host threads at once.  A call captured into a CUDA
 * graph takes its workspace from the graph's own memory, so graphs share
 * nothing with each other or with eager calls. */
int swin_block_rms_create(swin_block_rms_t *out, int C, float eps);

/* out = norm(x + residual) in bf16.
 *   x, residual, out_sum, out [rows, C] bf16, gamma [C] bf16
 * residual may be NULL (then out_sum must be NULL: s is x itself); out_sum
 * receives s and may be NULL.  out and out_sum may each be x or residual
 * itself (in place) but not the same buffer as each other, nor a partial
 * overlap of any other tensor.  EINVAL for NULL, misaligned (16 bytes) or
 * overlapping pointers or rows < 0; ECUDA for a launch failure.  rows = 0 is
 * a no-op. */
int swin_block_rms_forward(swin_block_rms_t h, const void *x, const void *residual, int rows, const void *gamma,
                           void *out_sum, void *out, swin_stream_t stream);

/* The same with the output in 8 bits: out8 [rows, C] e4m3 codes, scales
 * [rows] fp32 (16-byte aligned), neither overlapping any other tensor. */
int swin_block_rms_forward_q8(swin_block_rms_t h, const void *x, const void *residual, int rows, const void *gamma,
                              void *out_sum, void *out8, float *scales, swin_stream_t stream);

/* Gradients of sum(y dy) + sum(s dsum) with respect to s (equally x and
 * residual) and gamma:
 *   n = s r; a = dy gamma; dx = r (a - n mean_c(a n)) + dsum; dgamma = sum_rows dy n
 *   s [rows, C] bf16 (the forward's out_sum, or x), dy [rows, C] bf16, dsum
 *   [rows, C] bf16 (the gradient that reaches s past the norm; NULL = none)
 *   dx [rows, C] bf16, dgamma [C] fp32, overwritten
 * dgamma's sum over the rows is taken in a fixed order in fp32.  dx may be dy
 * or dsum itself, not a partial overlap and not s.  Errors as above, ENOMEM if the
 * workspace (partial sums of dgamma) cannot be allocated.  rows = 0 zeroes
 * dgamma. */
int swin_block_rms_backward(swin_block_rms_t h, const void *s, int rows, const void *gamma, const void *dy,
                            const void *dsum, void *dx, float *dgamma, swin_stream_t stream);

/* Number of kernel launches of the last call that launched (0 before). */
int swin_block_rms_last_launches(swin_block_rms_t h);

/* Frees the handle and its workspace (NULL is a no-op). */
int swin_block_rms_destroy(swin_block_rms_t h);

#ifdef __cplusplus
}
#endif

#endif /* SWIN_RMS_H */
