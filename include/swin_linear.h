/*
 * swin_block_linear -- a linear layer with its epilogue on one GB300 (sm_103a),
 * behind a plain C ABI: bias, activation and residual in the matrix product's
 * own kernel, an 8-bit form and a backward pass.  The block's MLP is two of
 * them (GELU; none with the residual), its projections and the merging step's
 * reduction one each.
 *
 * On tokens (rows) of C channels with N output channels:
 *   z = x W^T + b;  out = residual + act(z)
 * act: none, SiLU z / (1 + exp(-z)) or the exact GELU z Phi(z) of the block's
 * MLP.  bf16 tensors, the product on the tensor cores with fp32 accumulation,
 * everything behind it in fp32 and rounded once.  The kernels may start while
 * the kernel queued before them finishes (programmatic dependent launch) but
 * touch no memory before it has: a call needs no guarantee about its
 * parameters.  Conventions of swin_wattn.h: device pointers, asynchronous on
 * `stream`, caller-owned tensors, status codes SWIN_WATTN_*, no CPU fallback.
 */
#ifndef SWIN_LINEAR_H
#define SWIN_LINEAR_H

#include "swin_wattn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct swin_block_linear_s *swin_block_linear_t;

/* act of swin_block_linear_create. */
enum { SWIN_BLOCK_LINEAR_NONE = 0, SWIN_BLOCK_LINEAR_SILU = 1, SWIN_BLOCK_LINEAR_GELU = 2 };

/* C input and N output channels, multiples of 8, at most 65536.  *out receives
 * the handle (NULL on failure).  EINVAL for bad arguments, ENOMEM if the
 * handle's 4-byte device error word cannot be allocated.  The handle belongs to
 * the device that is current when it is created; calls with another current
 * device return EINVAL (without a device it can be created, and every call that
 * would launch returns ECUDA); creating it allocates, so not while a stream is
 * captured.  One handle may be used on several streams (its calls are ordered by
 * an event where they share its workspace, which grows to the largest call's and
 * then synchronises the device) but not from two host threads at once.  A call
 * captured into a CUDA graph takes its workspace from the graph's own memory, so
 * graphs share nothing with each other or with eager calls but the error word:
 * a graph is replayed only while its handle lives. */
int swin_block_linear_create(swin_block_linear_t *out, int C, int N, int act);

/* out = residual + act(x W^T + b).
 *   x [rows, C], W [N, C] (out x in), b [N] or NULL (zero), residual [rows, N] or
 *   NULL, z [rows, N] or NULL, out [rows, N], all bf16
 * z receives x W^T + b rounded to bf16 (what the backward pass of an activation
 * starts from; act is taken of the unrounded value, kept or not); with
 * SWIN_BLOCK_LINEAR_NONE it must be NULL.  out may be residual itself (in
 * place), not a partial overlap; out and z overlap no other tensor.  Every
 * pointer 16-byte aligned.  EINVAL for NULL, misaligned or overlapping pointers
 * or rows < 0 (or above 2^31 - 513); ENOMEM if the workspace (for few tiles: fp32
 * partial sums) cannot be allocated; ECUDA for a launch failure.  rows = 0 is a
 * no-op. */
int swin_block_linear_forward(swin_block_linear_t h, const void *x, int rows, const void *W, const void *b,
                              const void *residual, void *z, void *out, swin_stream_t stream);

/* The same from 8-bit inputs: x8 [rows, C] e4m3 with a scale a row, sx [rows]
 * fp32 (as swin_block_layernorm_forward_q8 and swin_block_rms_forward_q8 write
 * them), W8 [N, C] e4m3 with one fp32 scale per output channel, sw [N] (W ~ W8 *
 * sw): out = residual + act((x8 . W8) sx sw + b).  C must be a multiple of 16
 * (EUNSUPPORTED otherwise). */
int swin_block_linear_forward_q8(swin_block_linear_t h, const void *x8, const float *sx, int rows, const void *W8,
                                 const float *sw, const void *b, const void *residual, void *out,
                                 swin_stream_t stream);

/* Gradients of sum(out dy) (bf16 form; the residual's is dy itself):
 *   dz = dy act'(z); dx = dz W; dW = dz^T x; db = sum_rows dz
 *   x [rows, C], W [N, C], dy [rows, N], z [rows, N] (the forward's; NULL with
 *   SWIN_BLOCK_LINEAR_NONE, where dz = dy), dx [rows, C], dW [N, C], db [N], bf16
 * dx, dW and db are overwritten; each may be NULL (not computed: frozen
 * parameters, the model's first layer), but not dx and dW both, nor dW alone of
 * dW and db.  dz is rounded to bf16 before the products that read it; db adds
 * the unrounded values; every sum over rows is taken in a fixed order.  No
 * output overlaps an input or another output.  Errors as above; the workspace is
 * rows * N bf16 (N rounded up to a multiple of 64) where there is an activation,
 * plus fp32 partial sums.  rows = 0 zeroes the parameter gradients. */
int swin_block_linear_backward(swin_block_linear_t h, const void *x, int rows, const void *W, const void *z,
                               const void *dy, void *dx, void *dW, void *db, swin_stream_t stream);

/* Number of kernel launches of the last call that launched (0 before). */
int swin_block_linear_last_launches(swin_block_linear_t h);

/* Synchronises `stream` and reports an error the handle's kernels recorded since
 * the last call (SWIN_WATTN_ETIMEOUT), else SWIN_WATTN_OK. */
int swin_block_linear_sync_status(swin_block_linear_t h, swin_stream_t stream);

/* Frees the handle and its workspace (NULL is a no-op).  Synchronises the
 * device first. */
int swin_block_linear_destroy(swin_block_linear_t h);

#ifdef __cplusplus
}
#endif

#endif /* SWIN_LINEAR_H */
