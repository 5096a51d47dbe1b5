/*
 * mlp_block.h -- C ABI of the operators around the two products of a
 * transformer MLP block on MI355X (gfx950): layer norm and the linear layer
 * (matrix product with bias, activation and residual), forward and backward.
 * Part of the same library as mlp_chain.h; enums, error codes and
 * mlp_chain_last_error are that header's.
 *
 * With R rows (tokens), all matrices row-major and every 2-d operand with a
 * row stride of its own, in elements:
 *
 *   norm      mean_r = 1/H sum_c x[r,c]
 *             rstd_r = 1 / sqrt(1/H sum_c (x[r,c] - mean_r)^2 + eps)
 *             y[r,c] = (x[r,c] - mean_r) rstd_r weight[c] + bias[c]
 *   its       xhat = (x - mean) rstd,  g = dy weight
 *   gradient  dx = rstd (g - mean_c(g) - xhat mean_c(g xhat)) + dres
 *             dweight = sum_r dy xhat,  dbias = sum_r dy
 *
 *   linear    h = x W + bias           (z = h, saved on request)
 *             y = act(h) + residual
 *             act as in mlp_chain.h; swiglu reads W [K, 2N] and bias [2N]
 *             with the gate in columns 0..N-1 and up in N..2N-1
 *   its       dz = dy act'(z)          ([R, gN], g = 2 for swiglu, else 1)
 *   gradient  dx = dz W^T,  dW = x^T dz,  dbias = sum_r dz
 *             (the residual's gradient is dy itself)
 *
 * Numerics: inputs and outputs are fp16 or bf16, one type per handle; mean
 * and rstd are fp32.  Sums, statistics and accumulators are fp32 and every
 * output is rounded once (to nearest even), with one exception: dz is
 * rounded to the storage type before the two products of the linear
 * gradient, whose operands the matrix cores take in 16 bits; dbias sums it
 * unrounded.  Reductions have a fixed order: the same call gives the same
 * bits.  The outputs that the formulas make depend on a NaN or an infinity are
 * not finite either, the others are not touched by it; gelu_tanh's gradient at
 * an infinite z is its limit, dy or 0 (the formula has no value there).  fp32
 * bounds what is between: a dz or an output beyond the storage type is
 * infinite, and a row whose sum of (x - mean)^2 passes 3.4e38 (bf16) gets an
 * rstd of 0.
 *
 * Row counts: any R >= 0 per call, up to 2^24 and a linear handle's limit.  With R = 0
 * nothing is read and operands of R rows may be NULL; the forward passes
 * write nothing, the gradients of weights and biases are zero.
 *
 * Pointers are DEVICE pointers owned by the caller.  In the linear layer
 * they are 16-byte aligned, K and N are multiples of 8 and so are the row
 * strides (16-byte rows).  These are at most 2^36, but W's at most 2^23, and
 * x's, and dy's without an activation, at most the larger of 2^23 and
 * (2^31 - 2^24) / rows.  The norm takes any H >= 1, any row stride from H to
 * 2^36 and 2-byte aligned rows; 16-byte aligned rows with H a multiple of 8
 * run fastest.  y may be the residual's own buffer and a norm's dx may be dres's
 * (same row stride); no other outputs may overlap an operand.
 *
 * Streams, handles, errors: as in mlp_chain.h.  Every entry point but create
 * and destroy is asynchronous on `hip_stream`, launches kernels only (it may
 * be captured into a HIP graph) and depends on nothing from earlier calls.
 * A handle owns its workspace, so calls on one handle that may use it (every
 * call of a linear handle, the gradients of a norm) must be ordered on one
 * stream; separate handles are independent, and so are a norm's forward
 * passes, from any thread and on any stream.  destroy waits for the stream of
 * the handle's last call that may use the workspace.
 */
#ifndef MLP_BLOCK_H
#define MLP_BLOCK_H

#include <stdint.h>

#include "mlp_chain.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct mlp_norm* mlp_norm_t;
typedef struct mlp_linear* mlp_linear_t;

/* Create a layer norm over rows of H elements (1 <= H <= 2^22) with `eps`
 * (finite, >= 0) on the current HIP device.  `grad` != 0 allocates the
 * workspace of its gradient; a handle without it only runs forward.  Returns
 * NULL on error with mlp_chain_last_error() set. */
mlp_norm_t mlp_norm_create(int64_t H, int dtype, float eps, int grad);

/* y = norm(x) of `rows` rows.  weight and bias have H elements of the
 * storage type; NULL leaves out the scale or the shift.  mean and rstd
 * (fp32, `rows` each, 4-byte aligned) are written unless NULL; the gradient
 * needs both.  Returns MLP_EINVAL for bad pointers, sizes or strides,
 * MLP_EHIP if a launch fails. */
int mlp_norm_forward(mlp_norm_t h, int64_t rows, const void* x, int64_t ldx, const void* weight, const void* bias,
                     void* y, int64_t ldy, float* mean, float* rstd, void* hip_stream);

/* The gradient of mlp_norm_forward: dx from dy, x, weight (NULL: 1) and the
 * forward's mean and rstd; dres (NULL: none) is added to dx before its one
 * rounding -- the gradient that reaches x past the norm in a block with a
 * residual.  dweight and dbias (H elements each) are written unless NULL. */
int mlp_norm_backward(mlp_norm_t h, int64_t rows, const void* dy, int64_t lddy, const void* x, int64_t ldx,
                      const void* weight, const float* mean, const float* rstd, const void* dres, int64_t lddres,
                      void* dx, int64_t lddx, void* dweight, void* dbias, void* hip_stream);

/* Release the handle and its workspace.  NULL-safe. */
int mlp_norm_destroy(mlp_norm_t h);

/* Create a linear layer K -> N for calls of up to max_rows rows, on the
 * current HIP device.  max_rows >= 1, K and N positive multiples of 8, each
 * below 2^22; act and dtype from the enums of mlp_chain.h.  The workspace is
 * allocated here: the partials of split products (a few MB for single tokens,
 * at most 64 MB on 256 CUs) and, if `grad` != 0, what the gradient needs (dz
 * [max_rows, gN] with an activation); a handle without it only runs forward.
 * No weights are kept: one handle serves every layer of its sizes.  Returns
 * NULL on error with mlp_chain_last_error() set. */
mlp_linear_t mlp_linear_create(int64_t max_rows, int64_t K, int64_t N, int act, int dtype, int grad);

/* y = act(x W + bias) + residual for `rows` <= max_rows rows.  x [rows, K],
 * W [K, gN], bias [gN] or NULL, residual [rows, N] or NULL, y [rows, N];
 * z [rows, gN], unless NULL, receives h = x W + bias, which the gradient of
 * an activation needs.  The strides of absent operands are ignored.  Returns
 * MLP_EINVAL for bad pointers, sizes or strides, MLP_EHIP if a launch
 * fails. */
int mlp_linear_forward(mlp_linear_t h, int64_t rows, const void* x, int64_t ldx, const void* w, int64_t ldw,
                       const void* bias, const void* residual, int64_t ldres, void* y, int64_t ldy, void* z,
                       int64_t ldz, void* hip_stream);

/* The gradient of mlp_linear_forward: from dy [rows, N] and the saved z
 * (required unless act is none, then ignored) any of dx [rows, K] (needs w),
 * dw [K, gN] (needs x) and db [gN]; NULL outputs are not computed, and what
 * only they need may be NULL too. */
int mlp_linear_backward(mlp_linear_t h, int64_t rows, const void* dy, int64_t lddy, const void* x, int64_t ldx,
                        const void* w, int64_t ldw, const void* z, int64_t ldz, void* dx, int64_t lddx, void* dw,
                        int64_t lddw, void* db, void* hip_stream);

/* Release the handle and its workspace.  NULL-safe. */
int mlp_linear_destroy(mlp_linear_t h);

/* The plan a call of `rows` rows makes on a GPU with `cus` compute units for
 * pass 0 (x W), 1 (dz W^T alone), 2 (x^T dz alone), 3 or 4 (dz W^T and x^T dz
 * of a gradient that has both, which run in one launch), computed on the host
 * alone: fills the first min(n, 9) of
 *   { config id, parts of a split tile's reduction, BM, BN, tile rows, tile
 *     columns, 64-deep slabs per part, workspace bytes of the partials, tiles
 *     computed whole although the others are split }.
 * Returns MLP_EINVAL for sizes mlp_linear_create would reject, an unknown
 * pass, cus < 8, a NULL array or n < 3. */
int mlp_linear_plan(int64_t rows, int64_t K, int64_t N, int act, int pass, int cus, int64_t* plan, int n);

/* Test and measurement hook: run `pass` of the handle's later calls with tile
 * configuration `config_id` and the reduction of the tiles of the last, partial
 * round in at most `split` parts (0 or 1: one); config_id -1 and split 0 restore
 * the planner's choice.  Passes 3 and 4 share the configuration set last; a
 * forced pass 1 or 2 gives both products launches of their own.  A call whose
 * partials exceed the handle's workspace is then refused.  Returns
 * MLP_EINVAL for a NULL handle, a configuration the pass does not have or a
 * split outside 0..32. */
int mlp_linear_debug_set_plan(mlp_linear_t h, int pass, int config_id, int split);

#ifdef __cplusplus
}
#endif

#endif /* MLP_BLOCK_H */
