/*
 * onebit_layers.h -- C ABI of the layer operators that produce the gradients 1-bit Adam exchanges:
 * layer norm, the linear layer with its fused epilogue, and activation checkpoints held in 8 bits.
 *
 * Each worker of the data-parallel method runs a forward and a backward pass and hands its gradients,
 * in the optimizer's gradient type, to the steps of onebit_adam.h.  These calls are the feed-forward
 * half of a transformer layer in that form.  They have no counterpart on the method's pages.
 *
 * Conventions (those of onebit_adam.h):
 *   - `stream` is a cudaStream_t (NULL = legacy default stream).  Calls enqueue work on it and return
 *     without synchronising; every buffer must stay valid until the stream has passed the call.
 *     Calls on different streams are independent as long as their outputs and workspaces are.
 *   - Calls run on the calling thread's current device, which has to be the buffers' and the stream's.
 *   - A matrix is row-major with unit column stride: element (r, c) is at base + r*ld + c, with the
 *     row stride ld >= columns in elements.  Bases may have any alignment that the type needs, and
 *     ld any value; rows that start on 16-byte boundaries take the wide accesses (checkpoints: on 32-byte
 *     boundaries; layer norm: where gamma and beta lie on 16 bytes too).
 *   - dtype is onebit_dtype_t and names the type of x, y, dy, dx, residual and add.  Parameters that
 *     the optimizer holds in fp32 (gamma, beta, bias) are read in fp32; the linear layer's weight is
 *     read in dtype, as the 16-bit copy that a mixed-precision step makes of it.
 *   - Sums, statistics and products are accumulated in fp32; each output is rounded once.
 *   - Outputs must be disjoint from the inputs and from each other (ONEBIT_ERR_INVALID_ARG).
 *   - rows may be 0 (gradients of parameters are then 0); a width must be at least 1.
 *   - A failed check enqueues nothing, and leaves a message for onebit_layers_last_error().
 *   - Results do not depend on the grid or on timing: every sum has a fixed order.
 */
#ifndef ONEBIT_LAYERS_H
#define ONEBIT_LAYERS_H

#include "onebit_adam.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  ONEBIT_ACT_NONE = 0,
  ONEBIT_ACT_RELU = 1,      /* max(z, 0); its derivative at 0 is 0 */
  ONEBIT_ACT_GELU = 2,      /* z * Phi(z), Phi the standard normal distribution function */
  ONEBIT_ACT_GELU_TANH = 3  /* z/2 * (1 + tanh(sqrt(2/pi) * (z + 0.044715 z^3))) */
} onebit_activation_t;

/* ---- Activation checkpoints in 8 bits ----
 *
 * A matrix x of `cols` columns is held as int8 codes (rows*cols, contiguous) and fp32 scales
 * (rows*ceil(cols/64), contiguous): 64 consecutive columns of a row share one scale.  With
 * a = max |x| over the block, in fp32:
 *   scale = a / 127,  code = round_to_nearest_even(x * (127 / a)),  value = code * scale.
 * A block with a < 2^-120 has scale 0 and codes 0.  A block that holds an infinity or a NaN has scale
 * NaN and codes 0, so that all of it reads back as NaN. */
#define ONEBIT_CHECKPOINT_BLOCK 64

onebit_status_t onebit_checkpoint_compress(const void* x, int64_t ldx, int32_t dtype, int64_t rows, int64_t cols,
                                           int8_t* codes, float* scales, onebit_stream_t stream);
/* x = activation(value), in dtype. */
onebit_status_t onebit_checkpoint_restore(const int8_t* codes, const float* scales, int64_t rows, int64_t cols,
                                          int32_t activation, void* x, int64_t ldx, int32_t dtype,
                                          onebit_stream_t stream);

/* ---- Layer norm over the columns of each row ----
 *
 *   mean = sum(x)/cols;  rstd = 1/sqrt(sum((x-mean)^2)/cols + eps);  y = (x-mean)*rstd*gamma + beta
 * x, y: rows x cols of dtype (f32, f16 or bf16).  gamma, beta: cols fp32.  mean, rstd: rows fp32.
 * codes, scales: NULL, or the 8-bit checkpoint of x, written in the same pass. */
onebit_status_t onebit_layer_norm_forward(const void* x, int64_t ldx, int32_t dtype, int64_t rows, int64_t cols,
                                          const float* gamma, const float* beta, float eps, void* y, int64_t ldy,
                                          float* mean, float* rstd, int8_t* codes, float* scales,
                                          onebit_stream_t stream);

/* Bytes of device workspace that onebit_layer_norm_backward needs (16-byte aligned). */
onebit_status_t onebit_layer_norm_backward_workspace(int64_t rows, int64_t cols, size_t* bytes);

/* With xhat = (x-mean)*rstd and g = dy*gamma:
 *   dx = rstd*(g - sum(g)/cols - xhat*sum(g*xhat)/cols) [+ add];
 *   dgamma = sum over rows of dy*xhat;  dbeta = sum over rows of dy
 * The layer's input is x (with codes = scales = NULL) or its 8-bit checkpoint (x = NULL).  add: NULL,
 * or a second gradient of the layer's input (a residual path's), joined in fp32.  dgamma, dbeta: cols
 * values of grad_dtype. */
onebit_status_t onebit_layer_norm_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                                           const int8_t* codes, const float* scales, int32_t dtype, int64_t rows,
                                           int64_t cols, const float* gamma, const float* mean, const float* rstd,
                                           const void* add, int64_t ldadd, void* dx, int64_t lddx, void* dgamma,
                                           void* dbeta, int32_t grad_dtype, void* workspace, size_t workspace_bytes,
                                           onebit_stream_t stream);

/* ---- The linear layer ----
 *
 * Forward:  z = x w^T + bias;  y = activation(z) + residual.
 * x: rows x in, w: out x in, residual and y: rows x out, all of dtype f16 or bf16 (f32 is
 * ONEBIT_ERR_UNSUPPORTED); bias: out fp32 or NULL; residual may be NULL.  codes, scales: NULL, or the
 * 8-bit checkpoint of z (rows x out), made from the fp32 z in the product's epilogue. */
typedef struct {
  const void* x;
  int64_t ldx;
  const void* w;
  int64_t ldw;
  const float* bias;
  const void* residual;
  int64_t ldr;
  void* y;
  int64_t ldy;
  int8_t* codes;
  float* scales;
  int64_t rows, in, out;
  int32_t dtype;
  int32_t activation;
} onebit_linear_t;

/* Bytes of device workspace (256-byte aligned) that this call needs: 0 where rows lie on 16 bytes and the contraction
 * is not cut.  (onebit_linear_backward needs some also for an activation or a checkpoint behind dw, and for db of more
 * than 512 rows.) */
onebit_status_t onebit_linear_forward_workspace(const onebit_linear_t* a, size_t* bytes);
onebit_status_t onebit_linear_forward(const onebit_linear_t* a, void* workspace, size_t workspace_bytes,
                                      onebit_stream_t stream);

/* Backward of y = activation(v) w^T + bias with respect to v, w and bias, given dy:
 *   dx = (dy w) * activation'(v) [+ add];  dw = dy^T activation(v);  db = sum over rows of dy
 * v, the value before the activation that precedes the product, is x (codes = scales = NULL) or its
 * 8-bit checkpoint (x = NULL); with ONEBIT_ACT_NONE v is the product's input itself.  An
 * activation(v) or a value of a checkpoint that has to be computed is rounded to dtype before it enters
 * the product for dw, as the forward pass rounded what it multiplied w with: dw in fp32 is the fp32 sum
 * of those products, and good to dtype's digits as the derivative at an unrounded activation(v).
 * dy: rows x out, dx and add: rows x in, of dtype; dw: out x in contiguous, db: out, of grad_dtype.
 * dx, dw and db may each be NULL (not wanted); x and codes may both be NULL when only dx without an
 * activation, or only db, is wanted. */
typedef struct {
  const void* dy;
  int64_t lddy;
  const void* x;
  int64_t ldx;
  const int8_t* codes;
  const float* scales;
  const void* w;
  int64_t ldw;
  const void* add;
  int64_t ldadd;
  void* dx;
  int64_t lddx;
  void* dw;
  void* db;
  int64_t rows, in, out;
  int32_t dtype;
  int32_t activation;
  int32_t grad_dtype;
} onebit_linear_grad_t;

onebit_status_t onebit_linear_backward_workspace(const onebit_linear_grad_t* a, size_t* bytes);
onebit_status_t onebit_linear_backward(const onebit_linear_grad_t* a, void* workspace, size_t workspace_bytes,
                                       onebit_stream_t stream);

/* ---- Status ----
 *
 * Synchronise `stream` and report the device's sticky flag: ONEBIT_OK, or ONEBIT_ERR_CUDA when some
 * product gave up waiting (about one second) for its own asynchronous copies and stopped early; its
 * outputs are then not meaningful.  The CUDA context stays usable. */
onebit_status_t onebit_layers_get_status(onebit_stream_t stream);
/* Clear the flag (enqueued on `stream`). */
onebit_status_t onebit_layers_clear_status(onebit_stream_t stream);
/* Test hook, of the whole process: with ONEBIT_FAULT_STALL_COPIES the products of the following calls
 * wait for `value` bytes (1..2^19) that no copy delivers, so that their limited waits run out.
 * ONEBIT_FAULT_NONE turns it off.  Nothing here makes the GPU fault. */
onebit_status_t onebit_layers_set_fault_injection(int32_t kind, int64_t value);

/* Message of the last call of this header that failed on the calling thread ("" if none). */
const char* onebit_layers_last_error(void);

#ifdef __cplusplus
}
#endif
#endif /* ONEBIT_LAYERS_H */
