// residual_norm.cu -- the residual sum with the norms around it: a block's output through its norm, dropout and gate
// onto the residual stream, and the norm before the next block, forward and backward with the parameters' gradients.
// See include/onebit_layers.h for the formulas.
#include "residual_norm.cuh"

namespace onebit {
namespace layers {

// (in files of their own)
extern template cudaError_t rn_forward<float>(ResidualForward, cudaStream_t);
extern template cudaError_t rn_backward<float>(ResidualBackward, const ParamGrads&, int32_t, char*, int64_t*, cudaStream_t, bool);
extern template cudaError_t rn_forward<__half>(ResidualForward, cudaStream_t);
extern template cudaError_t rn_backward<__half>(ResidualBackward, const ParamGrads&, int32_t, char*, int64_t*, cudaStream_t, bool);
extern template cudaError_t rn_forward<__nv_bfloat16>(ResidualForward, cudaStream_t);
extern template cudaError_t rn_backward<__nv_bfloat16>(ResidualBackward, const ParamGrads&, int32_t, char*, int64_t*, cudaStream_t, bool);

namespace {

onebit_status_t shape_ok(int64_t rows, int64_t cols, int32_t dtype, int32_t norm) {
  if (rows < 0 || cols < 1) return fail(ONEBIT_ERR_INVALID_ARG, "rows or columns out of range");
  if (rows > kMaxRows || cols > kMaxCols) return fail(ONEBIT_ERR_UNSUPPORTED, "more than 2^31 rows or 2^24 columns");
  if (!dtype_ok(dtype)) return fail(ONEBIT_ERR_INVALID_ARG, "dtype is not one of f32, f16, bf16");
  if (norm != ONEBIT_NORM_LAYER && norm != ONEBIT_NORM_RMS) return fail(ONEBIT_ERR_INVALID_ARG, "unknown norm");
  return ONEBIT_OK;
}
bool all_aligned(std::initializer_list<const void*> p, uintptr_t a) {
  for (const void* q : p)
    if (!aligned(q, a)) return false;
  return true;
}

onebit_status_t forward_ok(const onebit_residual_norm_t& a, Dropout* drop) {
  onebit_status_t st = shape_ok(a.rows, a.cols, a.dtype, a.norm);
  if (st != ONEBIT_OK) return st;
  if (!(a.eps >= 0.0f)) return fail(ONEBIT_ERR_INVALID_ARG, "eps is negative or NaN");
  st = make_dropout(drop, a.p, a.key, a.site);
  if (st != ONEBIT_OK) return st;
  if (a.ldx < a.cols || (a.block && (a.ldblock < a.cols || a.lds < a.cols)) || (a.gamma && a.ldy < a.cols))
    return fail(ONEBIT_ERR_INVALID_ARG, "a row stride below the columns");
  if (a.rows == 0) return ONEBIT_OK;
  const bool layer = a.norm == ONEBIT_NORM_LAYER;
  if (!a.block && !a.gamma) return fail(ONEBIT_ERR_INVALID_ARG, "neither a block nor a norm");
  if (!a.block && (a.block_gamma || a.gate || drop->threshold))
    return fail(ONEBIT_ERR_INVALID_ARG, "a norm, gate or dropout of a block that is not there");
  if (!a.block != !a.s) return fail(ONEBIT_ERR_INVALID_ARG, "s is there where the block is, not else");
  if ((layer && a.gamma) != !!a.beta || (layer && a.block_gamma) != !!a.block_beta)
    return fail(ONEBIT_ERR_INVALID_ARG, "a layer norm has gamma and beta, an RMS norm gamma alone");
  if (!a.x || !a.gamma != !a.y || !a.gamma != !a.rstd || (layer && a.gamma) != !!a.mean || !a.block_gamma != !a.block_rstd ||
      (layer && a.block_gamma) != !!a.block_mean)
    return fail(ONEBIT_ERR_INVALID_ARG, "a buffer is NULL, or given for a norm that is not there");
  if (!all_aligned({a.x, a.block, a.s, a.y}, (uintptr_t)dtype_size(a.dtype)) ||
      !all_aligned({a.gamma, a.beta, a.block_gamma, a.block_beta, a.gate, a.mean, a.rstd, a.block_mean, a.block_rstd}, 4))
    return fail(ONEBIT_ERR_INVALID_ARG, "a buffer is not aligned to its type");
  const int64_t e = dtype_size(a.dtype), v = a.cols * 4, t = a.rows * 4;
  if (!disjoint({matrix(a.x, a.rows, a.ldx, a.cols, e), matrix(a.block, a.rows, a.ldblock, a.cols, e), span_of(a.gamma, v), span_of(a.beta, v),
                 span_of(a.block_gamma, v), span_of(a.block_beta, v), span_of(a.gate, v), span_of(a.key, 16)},
                {matrix(a.s, a.rows, a.lds, a.cols, e), matrix(a.y, a.rows, a.ldy, a.cols, e), span_of(a.mean, t), span_of(a.rstd, t),
                 span_of(a.block_mean, t), span_of(a.block_rstd, t)}))
    return fail(ONEBIT_ERR_INVALID_ARG, "an output overlaps another buffer");
  return ONEBIT_OK;
}

onebit_status_t backward_ok(const onebit_residual_norm_grad_t& a, Dropout* drop) {
  onebit_status_t st = shape_ok(a.rows, a.cols, a.dtype, a.norm);
  if (st != ONEBIT_OK) return st;
  if (!dtype_ok(a.grad_dtype)) return fail(ONEBIT_ERR_INVALID_ARG, "grad_dtype is not one of f32, f16, bf16");
  st = make_dropout(drop, a.p, a.key, a.site);
  if (st != ONEBIT_OK) return st;
  const bool layer = a.norm == ONEBIT_NORM_LAYER, any = a.rows > 0;
  if ((a.dy && a.lddy < a.cols) || (a.ds && a.ldds < a.cols) || (a.s && a.lds < a.cols) || (a.block && a.ldblock < a.cols) || a.lddx < a.cols ||
      (a.dblock && a.lddblock < a.cols))
    return fail(ONEBIT_ERR_INVALID_ARG, "a row stride below the columns");
  if (!a.gamma != !a.dgamma || (layer && a.gamma) != !!a.dbeta || !a.block_gamma != !a.dblock_gamma || (layer && a.block_gamma) != !!a.dblock_beta ||
      !a.gate != !a.dgate)
    return fail(ONEBIT_ERR_INVALID_ARG, "a parameter's gradient is there where the parameter is, not else");
  if (a.block_beta && !(layer && a.block_gamma)) return fail(ONEBIT_ERR_INVALID_ARG, "block_beta belongs to a layer norm behind the block");
  if (layer && a.block_gamma && a.gate && !a.block_beta) return fail(ONEBIT_ERR_INVALID_ARG, "dgate needs block_beta");
  if (any) {
    if (!a.dx || !a.gamma != !a.dy || (!a.gamma && !a.ds) || (a.gamma && !a.s))
      return fail(ONEBIT_ERR_INVALID_ARG, "dx, s and dy with gamma, or ds without, are needed");
    if ((a.block_gamma || a.gate) && !a.block) return fail(ONEBIT_ERR_INVALID_ARG, "the gradients of the block's norm and gate need the block");
    if (!a.dblock && (a.block_gamma || a.gate || drop->threshold))
      return fail(ONEBIT_ERR_INVALID_ARG, "a norm, gate or dropout of a block that is not there");
    if (!a.gamma != !a.rstd || (layer && a.gamma) != !!a.mean || !a.block_gamma != !a.block_rstd || (layer && a.block_gamma) != !!a.block_mean)
      return fail(ONEBIT_ERR_INVALID_ARG, "statistics are NULL, or given for a norm that is not there");
  }
  const uintptr_t ga = (uintptr_t)dtype_size(a.grad_dtype);
  if (!all_aligned({a.dy, a.ds, a.s, a.block, a.dx, a.dblock}, (uintptr_t)dtype_size(a.dtype)) ||
      !all_aligned({a.gamma, a.block_gamma, a.block_beta, a.gate, a.mean, a.rstd, a.block_mean, a.block_rstd}, 4) ||
      !all_aligned({a.dgamma, a.dbeta, a.dblock_gamma, a.dblock_beta, a.dgate}, ga))
    return fail(ONEBIT_ERR_INVALID_ARG, "a buffer is not aligned to its type");
  return ONEBIT_OK;
}

cudaError_t backward(const onebit_residual_norm_grad_t& a, const Dropout& drop, char* workspace, int64_t* used, cudaStream_t s, bool run) {
  const ResidualBackward b{a.dy, a.lddy, a.ds, a.ldds, a.s, a.lds, a.block, a.ldblock, a.gamma, a.block_gamma, a.block_beta, a.gate, drop, a.mean, a.rstd,
                       a.block_mean, a.block_rstd, a.dx, a.lddx, a.dblock, a.lddblock, a.rows, (int)a.cols, (int)ceil_div(a.cols, 8),
                       a.norm == ONEBIT_NORM_LAYER, 1.0f / (float)a.cols, a.scale, nullptr, nullptr};
  const ParamGrads g{a.dgamma, a.dbeta, a.dblock_gamma, a.dblock_beta, a.dgate};
  return a.dtype == ONEBIT_F32   ? rn_backward<float>(b, g, a.grad_dtype, workspace, used, s, run)
         : a.dtype == ONEBIT_F16 ? rn_backward<__half>(b, g, a.grad_dtype, workspace, used, s, run)
                                 : rn_backward<__nv_bfloat16>(b, g, a.grad_dtype, workspace, used, s, run);
}

}  // namespace
}  // namespace layers
}  // namespace onebit

using namespace onebit::layers;

extern "C" onebit_status_t onebit_residual_norm_forward(const onebit_residual_norm_t* p, onebit_stream_t stream) {
  if (!p) return fail(ONEBIT_ERR_INVALID_ARG, "the arguments are NULL");
  const onebit_residual_norm_t& a = *p;
  Dropout drop{};
  const onebit_status_t st = forward_ok(a, &drop);
  if (st != ONEBIT_OK || a.rows == 0) return st;
  const ResidualForward f{a.x, a.ldx, a.block, a.ldblock, a.gamma, a.beta, a.block_gamma, a.block_beta, a.gate, drop, a.s, a.lds, a.y, a.ldy, a.mean, a.rstd,
                      a.block_mean, a.block_rstd, a.rows, (int)a.cols, (int)ceil_div(a.cols, 8), a.norm == ONEBIT_NORM_LAYER, 1.0f / (float)a.cols,
                      a.eps, a.scale};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = a.dtype == ONEBIT_F32 ? rn_forward<float>(f, s) : a.dtype == ONEBIT_F16 ? rn_forward<__half>(f, s) : rn_forward<__nv_bfloat16>(f, s);
  return e == cudaSuccess ? ONEBIT_OK : cuda_fail(e, "onebit_residual_norm_forward");
}

extern "C" onebit_status_t onebit_residual_norm_backward_workspace(const onebit_residual_norm_grad_t* a, size_t* bytes) {
  if (!a) return fail(ONEBIT_ERR_INVALID_ARG, "the arguments are NULL");
  Dropout drop{};
  const onebit_status_t st = backward_ok(*a, &drop);
  if (st != ONEBIT_OK) return st;
  if (!bytes) return fail(ONEBIT_ERR_INVALID_ARG, "bytes is NULL");
  int64_t used = 0;
  backward(*a, drop, nullptr, &used, nullptr, false);
  *bytes = (size_t)used;
  return ONEBIT_OK;
}

extern "C" onebit_status_t onebit_residual_norm_backward(const onebit_residual_norm_grad_t* p, void* workspace, size_t workspace_bytes,
                                                         onebit_stream_t stream) {
  size_t need = 0;
  const onebit_status_t st = onebit_residual_norm_backward_workspace(p, &need);
  if (st != ONEBIT_OK) return st;
  const onebit_residual_norm_grad_t& a = *p;
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 16)))
    return fail(ONEBIT_ERR_WORKSPACE, "the workspace is too small or not 16-byte aligned");
  const int64_t e = dtype_size(a.dtype), g = a.cols * dtype_size(a.grad_dtype), v = a.cols * 4, t = a.rows * 4;
  if (!disjoint({matrix(a.dy, a.rows, a.lddy, a.cols, e), matrix(a.ds, a.rows, a.ldds, a.cols, e), matrix(a.s, a.rows, a.lds, a.cols, e),
                 matrix(a.block, a.rows, a.ldblock, a.cols, e), span_of(a.gamma, v), span_of(a.block_gamma, v), span_of(a.block_beta, v),
                 span_of(a.gate, v), span_of(a.key, 16), span_of(a.mean, t), span_of(a.rstd, t), span_of(a.block_mean, t), span_of(a.block_rstd, t)},
                {matrix(a.dx, a.rows, a.lddx, a.cols, e), matrix(a.dblock, a.rows, a.lddblock, a.cols, e), span_of(a.dgamma, g), span_of(a.dbeta, g),
                 span_of(a.dblock_gamma, g), span_of(a.dblock_beta, g), span_of(a.dgate, g), span_of(workspace, (int64_t)need)}))
    return fail(ONEBIT_ERR_INVALID_ARG, "an output overlaps another buffer");
  Dropout drop{};
  make_dropout(&drop, a.p, a.key, a.site);
  int64_t used = 0;
  const cudaError_t err = backward(a, drop, static_cast<char*>(workspace), &used, static_cast<cudaStream_t>(stream), true);
  return err == cudaSuccess ? ONEBIT_OK : cuda_fail(err, "onebit_residual_norm_backward");
}
