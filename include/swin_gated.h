/*
 * swin_block_gated -- the gated feed-forward block on one GB300 (sm_103a),
 * behind a plain C ABI: the gated form of the block's MLP (swin_block.h), with
 * the residual's addition, an 8-bit form and a backward pass.
 *
 * On tokens (rows) of C channels with hidden width F:
 *   g = x Wg^T + bg;  u = x Wu^T + bu;  h = act(g) * u
 *   out = residual + h Wd^T + bd
 * act: SWIN_BLOCK_GATED_SILU g / (1 + exp(-g)) or SWIN_BLOCK_GATED_GELU, the
 * exact GELU g Phi(g) of the block's MLP.  bf16 tensors, products on the tensor
 * cores with fp32 accumulation, activation and product in fp32; h is rounded to
 * bf16 once before the last product.  Both first projections, the activation
 * and the product are one kernel, the last projection with its bias and the
 * residual a second, sometimes with a third that joins tiles cut along F (the
 * bf16 form for C <= 128 and more than 128 rows is one kernel, and h stays on
 * chip, but for few rows with a long F; up to 128 rows take kernels of their
 * own).  The kernels may start while the kernel queued before them finishes
 * (programmatic dependent launch) but touch no memory before it has: a call
 * needs no guarantee about its parameters.  Conventions of swin_wattn.h: device
 * pointers, asynchronous on `stream`, caller-owned tensors, status codes
 * SWIN_WATTN_*, no CPU fallback.
 */
#ifndef SWIN_GATED_H
#define SWIN_GATED_H

#include "swin_wattn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct swin_block_gated_s *swin_block_gated_t;

/* act of swin_block_gated_create. */
enum { SWIN_BLOCK_GATED_SILU = 0, SWIN_BLOCK_GATED_GELU = 1 };

/* Parameters, device pointers, bf16: Wg, Wu [F, C], Wd [C, F] (out x in), bg, bu
 * [F], bd [C] (biases may be NULL: zero). */
typedef struct swin_block_gated_params {
    const void *Wg, *bg, *Wu, *bu, *Wd, *bd;
} swin_block_gated_params;

/* The 8-bit form's parameters: Wg8, Wu8 [F, C] in e4m3 with one fp32 scale per
 * output channel, sg, su [F] (Wg ~ Wg8 * sg); the rest as above, bf16. */
typedef struct swin_block_gated_params_q8 {
    const void *Wg8;
    const float *sg;
    const void *bg;
    const void *Wu8;
    const float *su;
    const void *bu;
    const void *Wd, *bd;
} swin_block_gated_params_q8;

/* The parameters' gradients, bf16 (the parameters' own type), overwritten.  A
 * bias gradient may be NULL: not computed. */
typedef struct swin_block_gated_grads {
    void *dWg, *dbg, *dWu, *dbu, *dWd, *dbd;
} swin_block_gated_grads;

/* C and F multiples of 8, at most 65536.  *out receives the handle (NULL on
 * failure).  EINVAL for bad arguments, ENOMEM if the handle's 4-byte device
 * error word cannot be allocated.  The handle belongs to the device that is
 * current when it is created; calls with another current device return EINVAL
 * (without a device it can be created, and every call that would launch
 * returns ECUDA); creating it allocates, so not while a stream is captured.  One
 * handle may be used on several streams (its calls are ordered by an event: they
 * share its workspace, which grows to the largest call's and then synchronises
 * the device) but not from two host threads at once.  A call captured into a CUDA
 * graph takes its workspace from the graph's own memory, so graphs share nothing
 * with each other or with eager calls but the error word: a graph is replayed
 * only while its handle lives. */
int swin_block_gated_create(swin_block_gated_t *out, int C, int F, int act);

/* out = residual + (act(x Wg^T + bg) * (x Wu^T + bu)) Wd^T + bd.
 * x, out [rows, C], residual [rows, C] or NULL.  out may be residual itself
 * (in place), not a partial overlap, and overlaps no other tensor.  Every
 * pointer 16-byte aligned.  EINVAL for NULL, misaligned or overlapping
 * pointers or rows < 0 (or above 2^31 - 513); ENOMEM if the workspace (rows * F bf16 with F rounded
 * up to a multiple of 64, for few tiles also fp32 partial sums) cannot be
 * allocated; ECUDA for a launch failure.  rows = 0 is a no-op. */
int swin_block_gated_forward(swin_block_gated_t h, const void *x, int rows, const swin_block_gated_params *p,
                             const void *residual, void *out, swin_stream_t stream);

/* The same from 8-bit inputs: x8 [rows, C] e4m3 with a scale a row, sx [rows]
 * fp32 (as swin_block_rms_forward_q8 writes them); g = (x8 . Wg8) sx sg + bg,
 * likewise u; h in bf16 (a row's scale is known only once all of it is) and so Wd
 * too (one matrix instruction takes operands of 16 or of 8 bits).  C must be a multiple of 16 (EUNSUPPORTED
 * otherwise). */
int swin_block_gated_forward_q8(swin_block_gated_t h, const void *x8, const float *sx, int rows,
                                const swin_block_gated_params_q8 *p, const void *residual, void *out,
                                swin_stream_t stream);

/* Gradients of sum(out dy) (bf16 form; the residual's is dy itself):
 *   dh = dy Wd; dg = dh u act'(g); du = dh act(g); dx = dg Wg + du Wu
 *   dWg = dg^T x; dWu = du^T x; dWd = dy^T h; dbg, dbu, dbd = the row sums of
 *   dg, du, dy
 * x, dy, dx [rows, C] bf16; g, u and h are recomputed from x (nothing of the
 * forward is kept); dg, du and h are rounded to bf16 before the products that
 * read them; every sum over rows is taken in a fixed order.  No output
 * overlaps an input or another output.  Errors as above; the workspace is 3 *
 * rows * F bf16, F rounded up as above, plus fp32 partial sums.  rows = 0 zeroes the parameter
 * gradients. */
int swin_block_gated_backward(swin_block_gated_t h, const void *x, int rows, const swin_block_gated_params *p,
                              const void *dy, void *dx, const swin_block_gated_grads *grads, swin_stream_t stream);

/* Number of kernel launches of the last call that launched (0 before). */
int swin_block_gated_last_launches(swin_block_gated_t h);

/* Synchronises `stream` and reports an error the handle's kernels recorded since
 * the last call (SWIN_WATTN_ETIMEOUT), else SWIN_WATTN_OK. */
int swin_block_gated_sync_status(swin_block_gated_t h, swin_stream_t stream);

/* Frees the handle and its workspace (NULL is a no-op).  Synchronises the
 * device first. */
int swin_block_gated_destroy(swin_block_gated_t h);

#ifdef __cplusplus
}
#endif

#endif /* SWIN_GATED_H */
