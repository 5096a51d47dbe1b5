/*
 * mlp_train.h -- C ABI of what makes a training step of the MLP block's
 * gradients on MI355X (gfx950): the softmax cross entropy of a vocabulary
 * head, forward and backward, without its logits; the norm of all gradients;
 * and an AdamW step over many tensors.  Part of the same library as
 * mlp_chain.h; enums, error codes and mlp_chain_last_error are that header's.
 *
 * With R rows (tokens) of x [R, H] and W [V, H], a row per word of the
 * vocabulary (an embedding's layout), matrices row-major, every 2-d operand
 * with a row stride of its own, in elements:
 *
 *   loss      z[r,v] = sum_h x[r,h] W[v,h]
 *             lse_r = log sum_v exp z[r,v]
 *             loss_r = lse_r - z[r,target_r]
 *   its       dz[r,v] = (dloss_r + dlse_r) exp(z[r,v] - lse_r) - dloss_r [v = target_r]
 *   gradient  dx = dz W,  dW = dz^T x
 *
 *   norm      norm = |unscale| sqrt(sum of all g^2)
 *             scale = unscale min(1, max_norm / norm), NaN if the norm is not finite
 *
 *   adamw     t = t + 1
 *             g = scale grad
 *             m = beta1 m + (1 - beta1) g
 *             v = beta2 v + (1 - beta2) g^2
 *             w = w (1 - lr decay) - lr / (1 - beta1^t) m / (sqrt(v / (1 - beta2^t)) + eps)
 *
 * Loss.  A row whose target is negative is left out: its x may hold anything
 * (in memory that can be read: where a call's rows fit one tile it is), its
 * loss, lse and dx are 0 and it adds nothing to dW.  A target of V or more
 * gives a loss and an lse of NaN; in the gradient its row is left out.  The
 * logits are never kept: the forward pass holds a maximum and a sum per row
 * and tile, the gradient makes the logits again, a piece of the vocabulary at
 * a time, as dz in the storage type.
 *
 * Numerics: x, W, dx, dW, gradients and weights are fp16 or bf16, one type
 * per handle; loss, lse and their gradients are fp32.  Sums and softmax are
 * fp32; every output is rounded once (to nearest even).  dz is rounded to the
 * storage type before its two products, whose operands the matrix cores take
 * in 16 bits, in units of the largest finite |dloss_r| or |dloss_r + dlse_r| of
 * the call (and in fp16 of 2^-14 of it, so that the rest of the vocabulary is not
 * lost: in fp16 dz below 2^-38 of that unit is).  Reductions have a fixed
 * order: the same call gives the same bits.  The gradient norm sums in 64
 * bits.  Outputs that the formulas make depend on a NaN or an infinity are not
 * finite either, the others are not touched by it.
 *
 * AdamW states are fp32 (32 bits) or floats of 8 bits: m in e4m3 (the OCP
 * type without infinities, largest 448), v in e5m2 (largest 57344), in blocks
 * of 256 elements of a tensor (the last one may be short), each with an fp32
 * scale, a power of two: the smallest one, but at least 2^-126, with which the
 * block's largest magnitude stays within the type (1 for a block of zeros).
 * The step itself takes m and v before they are rounded.  One step moves v by
 * less than half a step of 8 bits, so v is rounded up or down by chance, with a
 * mean of v, and to no less than the smallest number unless it is zero; its
 * random bits are a hash of `seed`, t, the tensor's number in the call and the
 * element's place.  m is rounded to nearest even, but by chance as well where
 * a step moves it by as little: with a beta1 above 15/16, and below 2^-6 of its
 * scale where the nearest is what it was, but for 0.  Elements that are not
 * finite are NaN in 8 bits and leave the scale alone.
 *
 * Row counts: any R >= 0 per call up to the handle's max_rows.  With R = 0
 * nothing is read, operands of R rows may be NULL and dW is zero.
 *
 * Pointers are DEVICE pointers owned by the caller.  x, W, dx and dW are
 * 16-byte aligned, H and the row strides are multiples of 8; V is any number.
 * Row strides are at most 2^36, but W's at most 2^23 and x's at most the
 * larger of 2^23 and (2^31 - 2^24) / rows.  The optimizer's tensors are
 * contiguous and need the alignment of their elements alone.  No output may
 * overlap an operand or another output.
 *
 * Streams, handles, errors: as in mlp_block.h.  Every entry point but create
 * and destroy is asynchronous on `hip_stream`, launches kernels only (it may
 * be captured into a HIP graph) and depends on nothing from earlier calls but
 * the caller's own tensors.  A handle owns its workspace, so calls on one
 * handle must be ordered on one stream; separate handles are independent.
 * destroy waits for the stream of the handle's last call.
 */
#ifndef MLP_TRAIN_H
#define MLP_TRAIN_H

#include <stdint.h>

#include "mlp_chain.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct mlp_loss* mlp_loss_t;
typedef struct mlp_grad_norm* mlp_grad_norm_t;
typedef struct mlp_adamw* mlp_adamw_t;

/* Create a cross entropy over V words from H-wide rows for calls of up to
 * max_rows rows, on the current HIP device.  1 <= max_rows <= 2^24, H a
 * positive multiple of 8 and V >= 1, each below 2^22, and no two of the three
 * with a product above 2^38.  The workspace is
 * allocated here: a copy of max_rows rows of x (calls that leave rows out
 * gather the others), 8 bytes per row and 128 words, 24 bytes per row, and if `grad` != 0 the
 * piece of dz (at most 256 MB, or 256 columns of max_rows rows where that is
 * more) and fp32 sums of dx; a handle without it only runs forward.  Returns
 * NULL on error with mlp_chain_last_error() set. */
mlp_loss_t mlp_loss_create(int64_t max_rows, int64_t H, int64_t V, int dtype, int grad);

/* loss and lse (fp32, `rows` each, 4-byte aligned; loss may be NULL) of x
 * [rows, H], W [V, H] and target (int64, `rows`, 8-byte aligned).  Returns
 * MLP_EINVAL for bad pointers, sizes or strides, MLP_EHIP if a launch fails. */
int mlp_loss_forward(mlp_loss_t h, int64_t rows, const void* x, int64_t ldx, const void* w, int64_t ldw,
                     const int64_t* target, float* loss, float* lse, void* hip_stream);

/* The gradient of mlp_loss_forward from its lse and dloss and dlse (fp32,
 * `rows` each; NULL: ones and zeros): dx [rows, H] and dw [V, H], written
 * unless NULL. */
int mlp_loss_backward(mlp_loss_t h, int64_t rows, const void* x, int64_t ldx, const void* w, int64_t ldw,
                      const int64_t* target, const float* lse, const float* dloss, const float* dlse, void* dx,
                      int64_t lddx, void* dw, int64_t lddw, void* hip_stream);

/* Release the handle and its workspace.  NULL-safe. */
int mlp_loss_destroy(mlp_loss_t h);

/* Test and measurement hook: the handle's later calls run the logits (product
 * 0) or the gradient's two products (1) with tile configuration `config_id` of
 * the linear layer (-1: the planner's), the latter with dx's reduction in at
 * most `split` parts (0: the planner's).  Returns MLP_EINVAL for a NULL handle,
 * a configuration the product does not have or a split outside 0..32. */
int mlp_loss_debug_set_plan(mlp_loss_t h, int product, int config_id, int split);

/* Create a gradient norm of tensors of `dtype` on the current HIP device. */
mlp_grad_norm_t mlp_grad_norm_create(int dtype);

/* The norm of `count` tensors together, grads[i] of 0 <= sizes[i] < 2^34
 * elements (NULL if none): norm (fp32, one element) and, unless NULL, scale (fp32, one
 * element), the factor that takes the gradients' loss scale out (`unscale`,
 * its magnitude within fp32's normal numbers; 1: none) and clips their norm to
 * max_norm (> 0, infinity: no clipping).  The arrays are read before the call
 * returns. */
int mlp_grad_norm_forward(mlp_grad_norm_t h, int64_t count, const int64_t* sizes, const void* const* grads,
                          double unscale, double max_norm, float* norm, float* scale, void* hip_stream);

int mlp_grad_norm_destroy(mlp_grad_norm_t h);

/* One tensor of an AdamW step. */
typedef struct {
    int64_t n;              /* elements, 0 <= n < 2^34 */
    void* w;                /* storage type */
    float* master;          /* fp32 weights: the step reads and writes these and w becomes their rounding; NULL: w itself */
    void* m;                /* fp32, or e4m3 bytes */
    void* v;                /* fp32, or e5m2 bytes */
    float* m_scale;         /* one per 256 elements; 32-bit states: ignored */
    float* v_scale;
    double decay;           /* weight decay, finite */
} mlp_adamw_tensor;

/* Create an AdamW optimizer of weights of `dtype` with states of `bits` (32
 * or 8) bits on the current HIP device.  0 <= beta1, beta2 < 1, eps 0 or at
 * least 2^-126 (a normal fp32 number) and finite.  With an eps of 0 an element
 * whose m and v are 0 becomes NaN, as the formula's 0 / 0. */
mlp_adamw_t mlp_adamw_create(int dtype, int bits, double beta1, double beta2, double eps, uint32_t seed);

/* One step of `count` tensors with grads[i] (storage type) of tensors[i].  t (int64, one element, 8-byte aligned, on the
 * device) counts the steps taken; the step's number is t + 1, in 1..2^31.
 * scale (fp32, one element on the device; NULL: 1) multiplies the gradients;
 * if it is NaN or infinite the step is left out: weights, states and t stay as
 * they are.  lr_scale (fp32, one element on the device; NULL: 1) multiplies lr
 * (finite), so that a captured step can follow a schedule.  The arrays are
 * read before the call returns. */
int mlp_adamw_step(mlp_adamw_t h, int64_t count, const mlp_adamw_tensor* tensors, const void* const* grads, double lr,
                   const float* lr_scale, const float* scale, int64_t* t, void* hip_stream);

int mlp_adamw_destroy(mlp_adamw_t h);

#ifdef __cplusplus
}
#endif

#endif /* MLP_TRAIN_H */
