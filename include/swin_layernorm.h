/*
 * swin_block_layernorm -- the block's layer norm as an operator of its own: with
 * the residual's addition in front of it (pre-norm) or behind it (residual
 * post-norm), an output in bf16 or in 8 bits with scales, and its backward
 * pass, on one GB300 (sm_103a), behind a plain C ABI.
 *
 * Per token (row) of C channels, in fp32 from bf16 tensors:
 *   s = x + residual (rounded to bf16; s = x without a residual)
 *   mu = mean_c s;  var = mean_c (s - mu)^2;  r = 1 / sqrt(var + eps);  n = (s - mu) r
 *   y = n gamma + beta
 * The statistics are sums of the row's differences from a pivot (the mean of its
 * first eight values; where that lies more than sqrt 2 standard deviations from the
 * row's mean, as beside a large channel, the sums are taken again about the mean),
 * not a difference of the large numbers mean s^2 and mu^2: a row of one value has n
 * = 0, a row far from zero loses nothing, and r's relative error is some 2^-21
 * (185 2^-24 at most, from chains of 40 additions) whatever the row holds.  The norm sees
 * the stored (rounded) sum, so that the backward pass, which starts from it,
 * differentiates the very function that ran.  A row holding an infinity or a NaN, or
 * whose first eight values or differences add up to more than 3.4e38, gives NaN; one
 * whose squared differences do has r = 0; with eps = 0, one whose channels are all
 * alike gives NaN or infinities, in the backward pass also in dgamma.  8-bit output: as
 * swin_block_rms_forward_q8 (swin_rms.h): scale = max(max_c |y|, 1e-30) / 448
 * per row, code = y / scale (both fp32 quotients) rounded to nearest even in
 * e4m3, NaN codes and a NaN scale for a row with a NaN.
 *
 * The block's own forward (swin_block.h) and swin_stage_norm have this norm with
 * eps = 1e-5 built in; this is what training and serving need beside them:
 * another eps, wider rows, the stored sum, the gradients.  Conventions of
 * swin_wattn.h: device pointers, asynchronous on `stream`, caller-owned tensors,
 * status codes SWIN_WATTN_*, no CPU fallback.
 */
#ifndef SWIN_LAYERNORM_H
#define SWIN_LAYERNORM_H

#include "swin_wattn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct swin_block_layernorm_s *swin_block_layernorm_t;

/* Rows of C channels (a multiple of 8, at most 16384) and eps >= 0 (finite).
 * *out receives the handle (NULL on failure).  EINVAL for bad arguments.  The
 * handle belongs to the device that is current at its first call that
 * launches; calls with another current device return EINVAL.  One handle may
 * be used on several streams (calls that need its workspace are ordered by an
 * event) but not from two host threads at once.  A call captured into a CUDA
 * graph takes its workspace from the graph's own memory, so graphs share
 * nothing with each other or with eager calls. */
int swin_block_layernorm_create(swin_block_layernorm_t *out, int C, float eps);

/* out = norm(x + residual) in bf16.
 *   x, residual, out_sum, out [rows, C] bf16, gamma, beta [C] bf16
 * beta may be NULL (zero).  residual may be NULL (then out_sum must be NULL: s
 * is x itself); out_sum receives s and may be NULL.  out and out_sum may each
 * be x or residual itself (in place) but not the same buffer as each other, nor
 * a partial overlap of any other tensor.  EINVAL for NULL, misaligned (16
 * bytes) or overlapping pointers or rows < 0; ECUDA for a launch failure.
 * rows = 0 is a no-op. */
int swin_block_layernorm_forward(swin_block_layernorm_t h, const void *x, const void *residual, int rows,
                                 const void *gamma, const void *beta, void *out_sum, void *out, swin_stream_t stream);

/* Residual post-norm: out = residual + norm(x), added in fp32 and rounded once
 * (x: the branch's output).  residual is required; out may be x or residual
 * itself.  Its gradients: the residual's is dy itself, x's and the parameters'
 * are those of swin_block_layernorm_backward with s = x and dsum = NULL. */
int swin_block_layernorm_forward_post(swin_block_layernorm_t h, const void *x, const void *residual, int rows,
                                      const void *gamma, const void *beta, void *out, swin_stream_t stream);

/* swin_block_layernorm_forward with the output in 8 bits: out8 [rows, C] e4m3
 * codes, scales [rows] fp32 (16-byte aligned), neither overlapping any other
 * tensor. */
int swin_block_layernorm_forward_q8(swin_block_layernorm_t h, const void *x, const void *residual, int rows,
                                    const void *gamma, const void *beta, void *out_sum, void *out8, float *scales,
                                    swin_stream_t stream);

/* Gradients of sum(y dy) + sum(s dsum) with respect to s (equally x and
 * residual), gamma and beta:
 *   a = dy gamma; dx = r (a - mean_c a - n mean_c(a n)) + dsum
 *   dgamma = sum_rows dy n; dbeta = sum_rows dy
 *   s [rows, C] bf16 (the forward's out_sum, or x), dy [rows, C] bf16, dsum
 *   [rows, C] bf16 (the gradient that reaches s past the norm; NULL = none)
 *   dx [rows, C] bf16, dgamma, dbeta [C] fp32, overwritten (dbeta may be NULL)
 * The sums over the rows are taken in a fixed order in fp32.  dx may be dy or
 * dsum itself, not a partial overlap and not s.  Errors as above, ENOMEM if the
 * workspace (partial sums of dgamma and dbeta) cannot be allocated.  rows = 0
 * zeroes dgamma and dbeta. */
int swin_block_layernorm_backward(swin_block_layernorm_t h, const void *s, int rows, const void *gamma, const void *dy,
                                  const void *dsum, void *dx, float *dgamma, float *dbeta, swin_stream_t stream);

/* Number of kernel launches of the last call that launched (0 before). */
int swin_block_layernorm_last_launches(swin_block_layernorm_t h);

/* Frees the handle and its workspace (NULL is a no-op). */
int swin_block_layernorm_destroy(swin_block_layernorm_t h);

#ifdef __cplusplus
}
#endif

#endif /* SWIN_LAYERNORM_H */
