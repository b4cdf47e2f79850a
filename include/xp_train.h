/*
 * xp_train.h — C ABI of the training operators around the ring allreduce:
 * layer norm forward and backward with the reduction of the weight's
 * gradient, the global norm of many gradients with its clip factor, and the
 * AdamW step over many tensors at once with states in 32 or 8 bits.
 *
 * A data-parallel step on virtual ranks runs: layer norm forward and backward
 * on each rank's rows (dgamma and dbeta come out in fp32, ready for
 * xp_ring_allreduce_virtual), the allreduce of the gradients, xp_grad_norm,
 * and xp_adamw_step, which takes the clip factor from device memory, so the
 * host waits for nothing in between.
 *
 * Conventions are those of xp.h: the same library (libxp.so), status codes,
 * xp_last_error(), streams (every call here is asynchronous on its stream;
 * NULL = the legacy default stream), argument errors without a launch, and
 * memory owned by the caller.  No call allocates except xp_group_create.
 * Every call but *_create, *_destroy and xp_group_get_step may be captured in a
 * CUDA graph.
 * Unlike the transfers, tensors here need only their element's alignment;
 * 16-byte aligned ones are faster.  Buffers a call writes must not overlap
 * any other buffer of the call, except where said.  (Matrices may be
 * side-by-side columns of one wider buffer; matrices whose rows are at
 * different distances and lie between one another's are refused.)
 */
#ifndef XP_TRAIN_H
#define XP_TRAIN_H

#include "xp.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------ layer norm */

/* Columns and rows the layer norm calls take at most (a row stays on chip). */
#define XP_LAYERNORM_MAX_COLS ((size_t)131072)
#define XP_LAYERNORM_MAX_ROWS ((size_t)1 << 28)

/* Per row of `cols` elements:
 *   mean = sum x / cols,  rstd = 1 / sqrt(sum (x - mean)^2 / cols + eps),
 *   y = (x - mean) * rstd * gamma + beta.
 * x and y are `dtype` (XP_F32 or XP_BF16), rows x_stride / y_stride elements
 * apart (>= cols); gamma and beta are `wdtype` (XP_F32 or XP_BF16), cols
 * each; either may be NULL (1 and 0).  mean and rstd (fp32, rows each) may be
 * NULL where no backward pass follows.  Statistics are fp32, over the row's
 * own values (two sums: the second about the mean; their terms have to stay
 * below 3.4e38, which deviations of 1e16 do in the longest rows); y is rounded
 * once.  y may be x itself when the strides are equal.  rows == 0 is a no-op. */
xp_status xp_layernorm_forward(const void* x, size_t x_stride, const void* gamma, const void* beta, void* y,
                               size_t y_stride, float* mean, float* rstd, size_t rows, size_t cols, float eps,
                               xp_dtype dtype, xp_dtype wdtype, xp_stream_t stream);

/* Bytes of workspace xp_layernorm_backward needs on the current device for
 * these sizes, at most (0 where rows or cols is 0). */
xp_status xp_layernorm_workspace(size_t rows, size_t cols, size_t* bytes);

/* With xhat = (x - mean) * rstd and a = dy * gamma (gamma NULL: 1), per row
 *   dx = rstd * (a - sum(a) / cols - xhat * sum(a * xhat) / cols),
 * and over the rows dgamma = sum dy * xhat, dbeta = sum dy (fp32, cols each;
 * both or neither may be NULL).  dy, x and dx are `dtype`, gamma `wdtype`,
 * mean and rstd what the forward pass gave.  accumulate != 0 adds to dgamma
 * and dbeta instead of overwriting them (rows == 0 then leaves them, and
 * zeroes them otherwise).  dx may be dy itself when the strides are equal.
 * `workspace` holds the rows' partial sums (16-byte aligned; its bytes are
 * checked against xp_layernorm_workspace); it is not needed, and may be NULL,
 * where dgamma is NULL.  Sums are fp32, in an order that depends on the sizes,
 * the type, the device, and whether rows and weights begin and end at multiples
 * of 16 bytes: equal calls on buffers alike in that give equal bits. */
xp_status xp_layernorm_backward(const void* dy, size_t dy_stride, const void* x, size_t x_stride, const void* gamma,
                                const float* mean, const float* rstd, void* dx, size_t dx_stride, float* dgamma,
                                float* dbeta, size_t rows, size_t cols, xp_dtype dtype, xp_dtype wdtype,
                                int accumulate, void* workspace, size_t workspace_bytes, xp_stream_t stream);

/* ------------------------------------------- groups of tensors and AdamW */

/* A group has one step count and one set of partial sums: calls on it follow
 * one another, on one stream or on streams that wait for each other.  Different
 * groups, and layer norm calls with workspaces of their own, may run at the same
 * time, and be made by different threads. */
typedef struct xp_group xp_group;   /* opaque, owned by the library */

/* One tensor of a group: device pointers, owned by the caller, valid until
 * xp_group_destroy.  State elements are fp32 (state_dtype XP_F32) or 8-bit
 * codes (XP_U8) with one scale byte per block of XP_STATE8_BLOCK elements
 * (ceil(count / 32) bytes; NULL for XP_F32). */
typedef struct {
  void* param;          /* param_dtype; NULL in every tensor: the group only serves xp_grad_norm */
  const void* grad;     /* grad_dtype */
  void* m;              /* first moment  */
  void* v;              /* second moment */
  uint8_t* m_scale;
  uint8_t* v_scale;
  void* copy;           /* XP_BF16 working copy of the updated weights, or NULL */
  size_t count;         /* elements; 0 is allowed */
  float weight_decay;   /* decoupled decay: p loses lr * weight_decay * p */
  int32_t reserved;     /* 0 */
} xp_tensor;

typedef struct {
  double beta1, beta2;  /* in [0, 1) */
  double eps;           /* > 0 */
  int32_t param_dtype;  /* XP_F32 or XP_BF16 */
  int32_t grad_dtype;   /* XP_F32 or XP_BF16 */
  int32_t state_dtype;  /* XP_F32, or XP_U8: 8-bit codes */
  uint32_t seed;        /* of the 8-bit states' rounding */
  uint64_t step;        /* steps already taken, XP_GROUP_MAX_STEP at most */
} xp_group_config;

/* An 8-bit state.  A block of 32 elements (block k holds elements 32 k ..
 * 32 k + 31 of its tensor) shares the scale byte E, the biased exponent of
 * the block's largest magnitude in fp32 (255: the block holds an infinity or
 * NaN and decodes as NaN).  A code's magnitude c > 0 stands for the fp32
 * number with the bit pattern (c + 8 E - K) << 20, that is an exponent and 3
 * mantissa bits; c = 0 is zero.  v uses all 8 bits (K = 247), m 7 bits below
 * a sign bit (K = 119).  Rounding to a code is stochastic: 20 bits (a 16-bit
 * hash h of the seed, the step and the element's position, as 16 h + 8) are
 * added to the fp32 pattern before it is cut, so a state's expected value is
 * kept although one step changes v by less than a code.  That holds from code 1
 * up, 2^-15 (m) and 2^-31 (v) of the block's power of two: below it an m becomes
 * 0 or code 1, and a v code 1, unless the v is below 2^-129 and the code stands
 * for 0.  The position of element i of tensor k is i + 32 times the blocks of
 * tensors 0 .. k - 1. */
#define XP_STATE8_BLOCK 32

/* The norm's outcome, in device memory (16-byte aligned). */
typedef struct {
  double sumsq;         /* sum of the squares of the gradients as stored */
  float norm;           /* grad_scale * sqrt(sumsq) */
  float scale;          /* what a step multiplies the gradients by: grad_scale, times max_norm / norm if norm > max_norm > 0 */
  int32_t nonfinite;    /* 1 if sumsq is an infinity or NaN */
  int32_t reserved[3];
} xp_grad_report;

/* Elements of a group at most, all tensors together, and the steps it may be
 * said to have taken (a step's number is exact in fp64). */
#define XP_GROUP_MAX_ELEMENTS ((size_t)1 << 40)
#define XP_GROUP_MAX_STEP ((uint64_t)1 << 52)

/* Make a group of `ntensors` tensors (1 <= ntensors <= 2^20) on the current
 * device: its tables (16 bytes per 2048 to 8192 elements, 80 per tensor) are
 * laid out once and reused by every call.  Errors: XP_ERR_INVALID (bad
 * argument), XP_ERR_CUDA, XP_ERR_INTERNAL (no host memory for the tables);
 * *out is untouched by all of them. */
xp_status xp_group_create(const xp_group_config* cfg, int ntensors, const xp_tensor* tensors, xp_group** out);

/* Synchronise the device, then free the group (not its tensors).  NULL is a
 * no-op. */
xp_status xp_group_destroy(xp_group* g);

/* Name other gradient buffers (a host array of ntensors device pointers, same
 * lengths and type) for the calls that follow on `stream`. */
xp_status xp_group_set_grads(xp_group* g, const void* const* grads, xp_stream_t stream);

/* The number of steps taken, set for the calls that follow on `stream`, or
 * read (waits for `stream`, and is refused while it is captured, which goes on). */
xp_status xp_group_set_step(xp_group* g, uint64_t step, xp_stream_t stream);
xp_status xp_group_get_step(xp_group* g, uint64_t* step, xp_stream_t stream);

/* The norm of all the group's gradients as one vector, into `report` (device
 * memory).  max_norm <= 0: no clipping.  accumulate != 0 adds the squares to
 * the report's sumsq first, so that the last of several groups' calls gives
 * the norm over all of them.  Squares are fp32: a gradient element beyond
 * 1.8e19 in magnitude overflows its square, and reads as not finite; one below
 * 1e-19 loses precision in it, and counts as 0 below 2e-23.  They are added in
 * fp32 within a warp's part of 2048 to 8192 elements and in fp64 beyond (in fp64
 * beyond eight elements where fp32 overflows), in an order that the lengths
 * alone decide.  sumsq is a NaN where a gradient is one, an infinity where one
 * overflows its square or is infinite, and finite otherwise. */
xp_status xp_grad_norm(xp_group* g, float grad_scale, float max_norm, int accumulate, xp_grad_report* report,
                       xp_stream_t stream);

/* xp_adamw_step's flags: leave weights, states and the step count as they are
 * if the report says nonfinite. */
#define XP_ADAMW_SKIP_NONFINITE 1

/* One AdamW step (t = steps taken + 1) on every tensor of the group, in fp32:
 *   g' = g * scale            (report->scale; report NULL: grad_scale)
 *   m = beta1 m + (1 - beta1) g',  v = beta2 v + (1 - beta2) g'^2
 *   p = p (1 - lr weight_decay) - lr / (1 - beta1^t) * m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
 * p and its copy are rounded to nearest even, 8-bit states as said above (the
 * step itself uses m and v before they are rounded).  The learning rate is
 * *lr_dev (device memory) if lr_dev is not NULL, for replayed graphs, else
 * lr.  The step count lives on the device and is advanced by the step. */
xp_status xp_adamw_step(xp_group* g, float lr, const float* lr_dev, float grad_scale, const xp_grad_report* report,
                        int flags, xp_stream_t stream);

/* The values 8-bit states stand for, as XP_F32 or XP_BF16 (exact in both):
 * `count` elements whose blocks follow one another, m_out from (m, m_scale)
 * and v_out from (v, v_scale); either pair's output may be NULL. */
xp_status xp_state8_decode(const uint8_t* m, const uint8_t* m_scale, const uint8_t* v, const uint8_t* v_scale,
                           size_t count, void* m_out, void* v_out, xp_dtype out_dtype, xp_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* XP_TRAIN_H */
