/*
 * onebit_layers.h -- C ABI of the layer operators that produce the gradients 1-bit Adam exchanges:
 * layer norm, the linear layer with its fused epilogue, the gated linear layer, dropout, the residual sum
 * with the norms around it, and activation checkpoints held in 8 bits.
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
  ONEBIT_ACT_GELU_TANH = 3, /* z/2 * (1 + tanh(sqrt(2/pi) * (z + 0.044715 z^3))) */
  ONEBIT_ACT_SILU = 4       /* z / (1 + exp(-z)): of the gated linear layer alone, refused elsewhere */
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

/* ---- The gated linear layer ----
 *
 * Forward:  [g | u] = z = x w^T + bias;  h = activation(g) * u.
 * x: rows x in; w: 2 inner x in, the gate's rows first, then those of the up projection; bias: 2 inner fp32 or
 * NULL; h: rows x inner; all but bias of dtype f16 or bf16 (f32 is ONEBIT_ERR_UNSUPPORTED).  What the backward pass
 * needs is kept as z (rows x 2 inner, of dtype) or as the 8-bit checkpoints of g and of u (rows x inner each, their own
 * blocks of 64 columns), made from the fp32 values, or not at all (z and the four of the checkpoints NULL). */
typedef struct {
  const void* x;
  int64_t ldx;
  const void* w;
  int64_t ldw;
  const float* bias;
  void* h;
  int64_t ldh;
  void* z;
  int64_t ldz;
  int8_t* gate_codes;
  float* gate_scales;
  int8_t* up_codes;
  float* up_scales;
  int64_t rows, in, inner;
  int32_t dtype;
  int32_t activation;
} onebit_gated_linear_t;

/* Bytes of device workspace (256-byte aligned) that this call needs. */
onebit_status_t onebit_gated_linear_forward_workspace(const onebit_gated_linear_t* a, size_t* bytes);
onebit_status_t onebit_gated_linear_forward(const onebit_gated_linear_t* a, void* workspace, size_t workspace_bytes,
                                            onebit_stream_t stream);

/* Backward of y = (activation(g) * u) w^T + bias with respect to z = [g | u], w and bias, given dy:
 *   dh = dy w;  dz = [dh * u * activation'(g) | dh * activation(g)];
 *   dw = dy^T (activation(g) * u);  db = sum over rows of dy
 * z is what the forward pass kept (gate_codes and the others NULL), or its checkpoints (z NULL).  dz is the dy of
 * onebit_linear_backward for the gated layer's own w and bias.  activation(g) * u is rounded to dtype before it
 * enters the product for dw, as the forward pass rounded h.
 * dy: rows x out; w: out x inner; dz: rows x 2 inner, of dtype; dw: out x inner contiguous, db: out, of grad_dtype.
 * dz, dw and db may each be NULL (not wanted); z and the checkpoints may all be NULL when only db is wanted. */
typedef struct {
  const void* dy;
  int64_t lddy;
  const void* z;
  int64_t ldz;
  const int8_t* gate_codes;
  const float* gate_scales;
  const int8_t* up_codes;
  const float* up_scales;
  const void* w;
  int64_t ldw;
  void* dz;
  int64_t lddz;
  void* dw;
  void* db;
  int64_t rows, inner, out;
  int32_t dtype;
  int32_t activation;
  int32_t grad_dtype;
} onebit_gated_linear_grad_t;

onebit_status_t onebit_gated_linear_backward_workspace(const onebit_gated_linear_grad_t* a, size_t* bytes);
onebit_status_t onebit_gated_linear_backward(const onebit_gated_linear_grad_t* a, void* workspace,
                                             size_t workspace_bytes, onebit_stream_t stream);

/* ---- Dropout ----
 *
 * Which elements are dropped follows from a counter-based generator, so that no mask is stored: the backward pass
 * draws it again (dx is dropout of dy, with the same p, key and site).
 *   t = round(65536 p);  an element stays where its 16 random bits, as a whole number, are at least t;
 *   y = x * (65536 / (65536 - t)) where it stays, 0 (whatever x) where it does not.
 * p is so held to steps of 1/65536; p < 0, NaN, or a p that rounds to 1 is ONEBIT_ERR_INVALID_ARG.
 * The random bits are Philox4x32-10 (Salmon et al., 2011) of the element's place: eight columns from 8 q on of
 * row r are group i = r * ceil(cols/8) + q, with the counter (i mod 2^32, i / 2^32, step mod 2^32, site) and the key
 * (seed mod 2^32, seed / 2^32).  Column 8 q + e has bits 16 (e mod 2) to 16 (e mod 2) + 15 of output word e/2.
 * key: two int64 in device memory, seed and step, read when the kernel runs (a captured graph meets new masks
 * when they change); may be NULL where t is 0.  site: the place in the model, so that one key serves a whole step. */
onebit_status_t onebit_dropout(const void* x, int64_t ldx, int32_t dtype, int64_t rows, int64_t cols, float p,
                               const int64_t* key, uint32_t site, void* y, int64_t ldy, onebit_stream_t stream);

/* ---- The residual sum with the norms around it ----
 *
 *   n = block, or norm(block) * block_gamma [+ block_beta] where block_gamma is given;
 *   s = x + scale * gate * dropout(n)           (gate NULL: 1; block NULL: s = x, which is not written);
 *   y = norm(s) * gamma [+ beta]                (gamma NULL: no y)
 * norm(v) = (v - mean) * rstd over the columns of a row.  ONEBIT_NORM_LAYER: mean = sum(v)/cols, rstd =
 * 1/sqrt(sum((v-mean)^2)/cols + eps), with beta (block_beta).  ONEBIT_NORM_RMS: mean = 0, rstd = 1/sqrt(sum(v^2)/cols
 * + eps), without.  Both norms are of one kind.  y is of the unrounded s.
 * x, block, s, y: rows x cols of dtype (f32, f16 or bf16).  gamma, beta, block_gamma, block_beta, gate: cols fp32.
 * mean, rstd, block_mean, block_rstd: rows fp32, outputs of the forward pass and inputs of the backward pass; the means
 * are NULL with ONEBIT_NORM_RMS, those of a norm that is not there too.  p, key and site as for onebit_dropout. */
typedef enum { ONEBIT_NORM_LAYER = 0, ONEBIT_NORM_RMS = 1 } onebit_norm_t;

typedef struct {
  const void* x;
  int64_t ldx;
  const void* block;
  int64_t ldblock;
  const float* gamma;
  const float* beta;
  const float* block_gamma;
  const float* block_beta;
  const float* gate;
  const int64_t* key;
  void* s;
  int64_t lds;
  void* y;
  int64_t ldy;
  float* mean;
  float* rstd;
  float* block_mean;
  float* block_rstd;
  int64_t rows, cols;
  int32_t dtype;
  int32_t norm;
  float eps;
  float scale;
  float p;
  uint32_t site;
} onebit_residual_norm_t;

onebit_status_t onebit_residual_norm_forward(const onebit_residual_norm_t* a, onebit_stream_t stream);

/* Given dy (gamma NULL: NULL) and ds, the gradient of s from the residual path (NULL: none; one of both is needed):
 *   shat = (s - mean) * rstd;  q = dy * gamma;
 *   t = rstd * (q [- sum(q)/cols] - shat * sum(q*shat)/cols) + ds;  dx = t;
 *   d = scale * t * the dropout's factor or 0;  e = d * gate;
 *   dblock = e, or behind a norm with bhat = (block - block_mean) * block_rstd and f = e * block_gamma:
 *            block_rstd * (f [- sum(f)/cols] - bhat * sum(f*bhat)/cols);
 *   dgamma = sum over rows of dy*shat;  dbeta = sum of dy;  dblock_gamma = sum of e*bhat;  dblock_beta = sum of e;
 *   dgate = sum of d*n                          (an element that dropout set to 0 adds nothing, whatever it was)
 * [..] with ONEBIT_NORM_LAYER.  s may be NULL without gamma, block without both block_gamma and gate.  dx: always.
 * dblock: NULL where there was no block (block, block_gamma, gate are then NULL and p is 0).  Each parameter's gradient,
 * cols values of grad_dtype, is there exactly where the parameter is: dgamma with gamma, dbeta with gamma and
 * ONEBIT_NORM_LAYER, dblock_gamma with block_gamma, dblock_beta likewise, dgate with gate (block_beta, as n's part, is
 * read for dgate alone and may be NULL without gate). */
typedef struct {
  const void* dy;
  int64_t lddy;
  const void* ds;
  int64_t ldds;
  const void* s;
  int64_t lds;
  const void* block;
  int64_t ldblock;
  const float* gamma;
  const float* block_gamma;
  const float* block_beta;
  const float* gate;
  const int64_t* key;
  const float* mean;
  const float* rstd;
  const float* block_mean;
  const float* block_rstd;
  void* dx;
  int64_t lddx;
  void* dblock;
  int64_t lddblock;
  void* dgamma;
  void* dbeta;
  void* dblock_gamma;
  void* dblock_beta;
  void* dgate;
  int64_t rows, cols;
  int32_t dtype;
  int32_t norm;
  int32_t grad_dtype;
  float scale;
  float p;
  uint32_t site;
} onebit_residual_norm_grad_t;

/* Bytes of device workspace (16-byte aligned) that this call needs. */
onebit_status_t onebit_residual_norm_backward_workspace(const onebit_residual_norm_grad_t* a, size_t* bytes);
onebit_status_t onebit_residual_norm_backward(const onebit_residual_norm_grad_t* a, void* workspace, size_t workspace_bytes,
                                              onebit_stream_t stream);

/* ---- Status ----
 *
 * Synchronise `stream` and report the device's sticky flag: ONEBIT_OK, or ONEBIT_ERR_CUDA when some
 * product gave up waiting (about one second) for its own asynchronous copies and stopped early, or a residual norm of
 * a row that several blocks share for a block's part of a sum; its outputs are then not meaningful.  The CUDA context
 * stays usable. */
onebit_status_t onebit_layers_get_status(onebit_stream_t stream);
/* Clear the flag (enqueued on `stream`). */
onebit_status_t onebit_layers_clear_status(onebit_stream_t stream);
/* Test hook, of the whole process: with ONEBIT_FAULT_STALL_COPIES the products of the following calls, and their
 * residual norms of rows that several blocks share, wait for `value` bytes (1..2^19) that nothing delivers, so
 * that their limited waits run out.
 * ONEBIT_FAULT_NONE turns it off.  Nothing here makes the GPU fault. */
onebit_status_t onebit_layers_set_fault_injection(int32_t kind, int64_t value);

/* Message of the last call of this header that failed on the calling thread ("" if none). */
const char* onebit_layers_last_error(void);

#ifdef __cplusplus
}
#endif
#endif /* ONEBIT_LAYERS_H */
