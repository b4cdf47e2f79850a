/*
 * xp_model.h — C ABI of the operators of a layer that trains and serves in 8
 * bits: the root-mean-square norm with the residual's addition and an output
 * in 8 bits, forward and backward; the encoding of matrices in 8 bits by blocks
 * of 128, and their decoding; the product of two such matrices; and the loss
 * that distils a teacher's top logits, forward and backward.
 *
 * A step of a model's last layer runs: xp_rmsnorm_forward (the sum, the norm
 * for the backward pass, the norm in 8 bits), xp_matmul8 with a weight that
 * xp_block8_encode made (the logits), xp_distill_forward and _backward,
 * xp_block8_encode of the gradient in both forms, xp_matmul8 twice (the
 * norm's gradient, and the weight's, in fp32 and added up over
 * micro-batches), xp_rmsnorm_backward.  The weights' gradients are fp32, ready
 * for xp_ring_allreduce_virtual, xp_grad_norm and xp_adamw_step.
 *
 * Conventions are those of xp_train.h: the same library (libxp.so), status
 * codes, xp_last_error(), streams (every call but xp_matmul8_status is
 * asynchronous on its stream; NULL = the legacy default stream), argument
 * errors without a launch, memory owned by the caller.  No call allocates, and
 * every call but xp_matmul8_status may be captured in a CUDA graph.  Matrices
 * are row-major, their rows a given number of elements apart.  Tensors need
 * their element's alignment, and 16 bytes are faster, except where said.
 * Buffers a call writes must not overlap any other buffer of the call, except
 * where said.  Calls may run at the same time, and be made by different
 * threads, where none writes what another reads or writes.
 */
#ifndef XP_MODEL_H
#define XP_MODEL_H

#include "xp.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Rows and columns of a matrix at most, and what rows are apart at most. */
#define XP_MODEL_MAX_ROWS ((size_t)1 << 28)
#define XP_MODEL_MAX_COLS ((size_t)1 << 20)
#define XP_MODEL_MAX_STRIDE ((size_t)1 << 36)

/* ------------------------------------------- matrices in 8 bits by blocks */

/* A matrix in 8 bits is a matrix of codes and one of scales.  A code is a sign,
 * 4 exponent bits e and 3 mantissa bits f (e4m3): (-1)^s 2^(e - 7) (1 + f / 8),
 * 2^-6 f / 8 where e is 0; 0x7f and 0xff are NaN, the largest is 448.  A block
 * is XP_BLOCK8 columns of one row (block_rows 1: gradients, activations), or of
 * 128 rows (block_rows 128: weights); the last of a row or column may have
 * fewer.  All of a block's codes are times 2^(E - 127) for its scale byte E:
 * the least E with max |x| <= 448 * 2^(E - 127), or 255, NaN, where the block
 * holds an infinity or a NaN (its codes are 0x7f then).  The scales of a matrix
 * of rows x cols are ceil(rows / block_rows) x ceil(cols / 128) bytes.
 * For xp_matmul8 codes begin at, and their rows are, multiples of 16 bytes
 * apart, scales 4 bytes; what lies between rows does not matter.  (Rows of
 * codes at multiples of 128 bytes are faster: a tenth less time with many rows
 * and columns.) */
#define XP_BLOCK8 128

/* Encode x (`dtype` XP_F32 or XP_BF16): x / 2^(E - 127) rounded to the nearest
 * code, ties to even.  codes (rows x cols) with scales, and codes_t with
 * scales_t, the encoding of x's transpose (cols x rows): its blocks run along
 * x's columns.  (With block_rows 128 it has the same codes, transposed.)
 * Either pair may be NULL, not both.  rows == 0 or cols == 0 is a no-op. */
xp_status xp_block8_encode(const void* x, size_t x_stride, size_t rows, size_t cols, xp_dtype dtype, int block_rows,
                           uint8_t* codes, size_t codes_stride, uint8_t* scales, size_t scales_stride, uint8_t* codes_t,
                           size_t codes_t_stride, uint8_t* scales_t, size_t scales_t_stride, xp_stream_t stream);

/* The values that codes stand for, as XP_F32 or XP_BF16: exact in both, except
 * below 2^-126 (bf16 rounds what it cannot hold) and where 256 * 2^120 would
 * be meant, an infinity. */
xp_status xp_block8_decode(const uint8_t* codes, size_t codes_stride, const uint8_t* scales, size_t scales_stride,
                           size_t rows, size_t cols, int block_rows, void* out, size_t out_stride, xp_dtype dtype,
                           xp_stream_t stream);

/* c = a b^T (m x n), or c + a b^T with accumulate != 0, of a (m x k) and b
 * (n x k) in 8 bits with blocks of a_block_rows and b_block_rows rows.  c is
 * XP_F32 or XP_BF16 (accumulate: XP_F32), at any alignment of its element.
 * Products are exact and summed in fp32 by the tensor cores, rounded once to
 * c's type; the order of the additions depends on m, n, k, and the device
 * alone: equal products give equal bits, wherever their rows lie.  A block whose
 * scale is 255 makes its rows of a, or its columns of c, NaN.  k == 0 gives
 * zeros, or leaves c. */
xp_status xp_matmul8(const uint8_t* a, size_t a_stride, const uint8_t* a_scales, size_t a_scales_stride, int a_block_rows,
                     const uint8_t* b, size_t b_stride, const uint8_t* b_scales, size_t b_scales_stride, int b_block_rows,
                     void* c, size_t c_stride, size_t m, size_t n, size_t k, xp_dtype c_dtype, int accumulate,
                     xp_stream_t stream);

/* Waits for the device.  XP_ERR_TIMEOUT if a product on the current device
 * ever gave up a wait between its own warps (after the spin timeout of xp.h, two
 * seconds, which has to be above 0.1 ms for them; what it had not summed by then
 * is NaN), else XP_OK.  (xp_abort does not stop a product.)  Not while a stream of the device is being captured: like
 * any call that waits for a device, it would end the capture. */
xp_status xp_matmul8_status(void);

/* ------------------------------------------------- root-mean-square norm */

/* Per row of `cols` elements, with h = x, or x + residual rounded to the type
 * (and stored in `added`) where residual is not NULL:
 *   rstd = 1 / sqrt(sum h^2 / cols + eps),   y = h * rstd * gamma.
 * x, residual, added and y are `dtype` (XP_F32 or XP_BF16), gamma `wdtype`
 * (NULL: 1).  y is rounded once.  y8 and y8_scales are y in 8 bits with
 * block_rows 1, encoded from its values before they are rounded to `dtype`.
 * y, y8 (with its scales) and rstd (fp32) may each be NULL; added is NULL
 * where residual is, and only there.  added may be x or residual itself, and y
 * may be x or residual itself where added is not the same one, at equal strides.
 * Sums are fp32 (elements of 1e16 and more overflow them).  rows == 0 is a
 * no-op. */
xp_status xp_rmsnorm_forward(const void* x, size_t x_stride, const void* residual, size_t residual_stride,
                             const void* gamma, void* added, size_t added_stride, void* y, size_t y_stride, uint8_t* y8,
                             size_t y8_stride, uint8_t* y8_scales, size_t y8_scales_stride, float* rstd, size_t rows,
                             size_t cols, float eps, xp_dtype dtype, xp_dtype wdtype, xp_stream_t stream);

/* Bytes of workspace xp_rmsnorm_backward needs on the current device for
 * these sizes (0 where rows or cols is 0). */
xp_status xp_rmsnorm_workspace(size_t rows, size_t cols, size_t* bytes);

/* With h the norm's input (x, or what the forward pass stored in `added`),
 * xhat = h * rstd and a = dy * gamma, per row
 *   dx = rstd * (a - xhat * sum(a * xhat) / cols) + dadded,
 * the gradient of x and of the residual alike; dadded (NULL: 0) is the
 * gradient that reaches h by itself.  Over the rows dgamma = sum dy * xhat
 * (fp32, cols; may be NULL); accumulate != 0 adds to it (rows == 0 then leaves
 * it, and zeroes it otherwise).  dy, h, dadded and dx are `dtype`, gamma
 * `wdtype`.  dx may be dy or dadded itself when the strides are equal.
 * `workspace` (16-byte aligned, its bytes are checked) is needed where dgamma
 * is not NULL or cols is above 8192.  Sums are fp32 in an order that the sizes, the types, the
 * alignment and the device alone decide. */
xp_status xp_rmsnorm_backward(const void* dy, size_t dy_stride, const void* h, size_t h_stride, const void* gamma,
                              const float* rstd, const void* dadded, size_t dadded_stride, void* dx, size_t dx_stride,
                              float* dgamma, size_t rows, size_t cols, xp_dtype dtype, xp_dtype wdtype, int accumulate,
                              void* workspace, size_t workspace_bytes, xp_stream_t stream);

/* ----------------------------------- distillation from top logits */

/* Entries per row at most. */
#define XP_DISTILL_MAX_TOP ((size_t)1024)

/* Per row of `vocab` logits z, with the teacher's `top` entries (ids, logits t):
 * q = softmax(z / T), p = softmax(t / T) over the row's entries,
 *   loss = T^2 sum_j p_j (log p_j - log q[ids_j]),   lse = log sum exp(z / T).
 * An entry whose id is not in [0, vocab) (-1, say) names no token and counts
 * for nothing; so does one whose t is -infinity.  An id may come more than
 * once: its entries each add to it.  A row without entries has loss 0 and lse
 * 0, whatever its logits.  z is `dtype` (XP_F32 or XP_BF16), ids int32,
 * t fp32, rows x top each, side by side; loss and lse fp32, lse may be NULL
 * where no backward pass follows.  (One entry is the cross entropy of a
 * label.)  Sums are fp32; logits over T that count have to be below 3e38 (masks of
 * the type's lowest value need not be, nor the teacher's, even where they are all
 * of a row's). */
xp_status xp_distill_forward(const void* logits, size_t logits_stride, const int32_t* ids, const float* teacher,
                             size_t rows, size_t vocab, size_t top, float temperature, float* loss, float* lse,
                             xp_dtype dtype, xp_stream_t stream);

/* dlogits = dloss T (q - p), the gradient of sum_i dloss_i loss_i, with q from
 * the forward pass's lse; rows without entries get zeros.  dlogits is `dtype`
 * and may be the logits themselves when the strides are equal.  Entries of one
 * id are added in their order. */
xp_status xp_distill_backward(const void* logits, size_t logits_stride, const int32_t* ids, const float* teacher,
                              const float* lse, const float* dloss, size_t rows, size_t vocab, size_t top,
                              float temperature, void* dlogits, size_t dlogits_stride, xp_dtype dtype,
                              xp_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* XP_MODEL_H */
