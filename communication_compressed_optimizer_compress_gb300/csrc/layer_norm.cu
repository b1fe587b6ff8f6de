// layer_norm.cu -- layer norm over the columns of each row, forward and backward, with the gradients
// of gamma and beta.  See include/onebit_layers.h for the formulas.
#include "layers_common.cuh"

namespace onebit {
namespace layers {
namespace {

constexpr int kLnThreads = 256;
constexpr int kLnWarps = kLnThreads / 32;

// Sum over the block, the same order on every call; every thread gets it.
__device__ __forceinline__ float block_sum(float v, float* red) {
  v = warp_sum(v);
  __syncthreads();  // red may still be read from the sum before
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = 0.0f;
#pragma unroll
  for (int w = 0; w < kLnWarps; ++w) t += red[w];
  return t;
}

// One block per row: the mean, then the squared distances from it, then the output.
template <typename T>
__global__ void __launch_bounds__(kLnThreads) k_ln_forward(const T* __restrict__ x, int64_t ldx, int64_t rows, int cols,
                                                           const float* __restrict__ gamma,
                                                           const float* __restrict__ beta, float eps,
                                                           T* __restrict__ y, int64_t ldy, float* __restrict__ mean_out,
                                                           float* __restrict__ rstd_out, int8_t* __restrict__ codes,
                                                           float* __restrict__ scales, int blocks) {
  __shared__ float red[kLnWarps];
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const T* xr = x + r * ldx;
    float s = 0.0f;
    for (int c = threadIdx.x; c < cols; c += kLnThreads) s += to_f(xr[c]);
    const float mean = block_sum(s, red) / (float)cols;
    s = 0.0f;
    for (int c = threadIdx.x; c < cols; c += kLnThreads) {
      const float d = to_f(xr[c]) - mean;
      s = fmaf(d, d, s);
    }
    const float rstd = 1.0f / sqrtf(block_sum(s, red) / (float)cols + eps);
    for (int c = threadIdx.x; c < cols; c += kLnThreads)
      y[r * ldy + c] = from_f<T>(fmaf((to_f(xr[c]) - mean) * rstd, gamma[c], beta[c]));
    if (threadIdx.x == 0) {
      mean_out[r] = mean;
      rstd_out[r] = rstd;
    }
    if (codes) {
      const int lane = threadIdx.x & 31;
      for (int b = threadIdx.x >> 5; b < blocks; b += kLnWarps) {
        const int c0 = b * kBlock + lane, c1 = c0 + 32;
        const float v0 = c0 < cols ? to_f(xr[c0]) : 0.0f, v1 = c1 < cols ? to_f(xr[c1]) : 0.0f;
        const BlockScale q = block_scale(warp_max_nan(max_nan(fabsf(v0), fabsf(v1))));
        if (c0 < cols) codes[r * cols + c0] = (int8_t)code_of(v0, q.inv);
        if (c1 < cols) codes[r * cols + c1] = (int8_t)code_of(v1, q.inv);
        if (lane == 0) scales[r * blocks + b] = q.scale;
      }
    }
  }
}

// The layer's input as the backward pass has it: the values themselves, or their 8-bit checkpoint.
template <typename T>
struct Input {
  const T* x;
  int64_t ldx;
  const int8_t* codes;
  const float* scales;
  int cols, blocks;
  __device__ __forceinline__ float at(int64_t r, int c) const {
    return codes ? value_of<T>(codes[r * cols + c], scales[r * blocks + c / kBlock]) : to_f(x[r * ldx + c]);
  }
};

template <typename T>
__global__ void __launch_bounds__(kLnThreads) k_ln_backward(const T* __restrict__ dy, int64_t lddy, Input<T> in,
                                                            int64_t rows, int cols, const float* __restrict__ gamma,
                                                            const float* __restrict__ mean,
                                                            const float* __restrict__ rstd, const T* __restrict__ add,
                                                            int64_t ldadd, T* __restrict__ dx, int64_t lddx) {
  __shared__ float red[kLnWarps];
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const float mu = mean[r], rs = rstd[r];
    float s1 = 0.0f, s2 = 0.0f;
    for (int c = threadIdx.x; c < cols; c += kLnThreads) {
      const float g = to_f(dy[r * lddy + c]) * gamma[c];
      s1 += g;
      s2 = fmaf(g, (in.at(r, c) - mu) * rs, s2);
    }
    s1 = block_sum(s1, red) / (float)cols;
    s2 = block_sum(s2, red) / (float)cols;
    for (int c = threadIdx.x; c < cols; c += kLnThreads) {
      const float g = to_f(dy[r * lddy + c]) * gamma[c];
      float d = rs * (g - s1 - (in.at(r, c) - mu) * rs * s2);
      if (add) d += to_f(add[r * ldadd + c]);
      dx[r * lddx + c] = from_f<T>(d);
    }
  }
}

// dgamma and dbeta: part[chunk][2][cols] over runs of kRun rows, then their sum in chunk order.
constexpr int kRun = 128;
template <typename T>
__global__ void __launch_bounds__(kLnThreads) k_ln_param_part(const T* __restrict__ dy, int64_t lddy, Input<T> in,
                                                              int64_t rows, int cols, const float* __restrict__ mean,
                                                              const float* __restrict__ rstd, float* __restrict__ part) {
  const int c = blockIdx.x * kLnThreads + threadIdx.x;
  if (c >= cols) return;
  for (int64_t ch = blockIdx.y; ch * kRun < rows; ch += gridDim.y) {
    const int64_t end = (ch + 1) * kRun < rows ? (ch + 1) * kRun : rows;
    float g = 0.0f, b = 0.0f;
    for (int64_t r = ch * kRun; r < end; ++r) {
      const float d = to_f(dy[r * lddy + c]);
      g = fmaf(d, (in.at(r, c) - mean[r]) * rstd[r], g);
      b += d;
    }
    part[(ch * 2) * cols + c] = g;
    part[(ch * 2 + 1) * cols + c] = b;
  }
}
template <typename G>
__global__ void __launch_bounds__(kLnThreads) k_ln_param_sum(const float* __restrict__ part, int64_t chunks, int cols,
                                                             G* __restrict__ dgamma, G* __restrict__ dbeta) {
  const int c = blockIdx.x * kLnThreads + threadIdx.x;
  if (c >= cols) return;
  float g = 0.0f, b = 0.0f;
  for (int64_t ch = 0; ch < chunks; ++ch) {
    g += part[(ch * 2) * cols + c];
    b += part[(ch * 2 + 1) * cols + c];
  }
  dgamma[c] = from_f<G>(g);
  dbeta[c] = from_f<G>(b);
}

int row_grid(int64_t rows) {
  const int64_t most = (int64_t)sm_count() * 8;
  return (int)(rows < most ? rows : most);
}

struct BackwardArgs {
  const void* dy;
  int64_t lddy;
  const void* x;
  int64_t ldx;
  const int8_t* codes;
  const float* scales;
  int64_t rows;
  int cols, blocks;
  const float *gamma, *mean, *rstd;
  const void* add;
  int64_t ldadd;
  void* dx;
  int64_t lddx;
  void *dgamma, *dbeta;
  int32_t grad_dtype;
  float* part;
};

template <typename T>
cudaError_t launch_backward(const BackwardArgs& a, cudaStream_t s) {
  const T* dy = static_cast<const T*>(a.dy);
  const Input<T> in{static_cast<const T*>(a.x), a.ldx, a.codes, a.scales, a.cols, a.blocks};
  const int64_t chunks = ceil_div(a.rows, kRun);
  const unsigned cgrid = (unsigned)ceil_div(a.cols, kLnThreads);
  if (a.rows > 0) {
    k_ln_backward<T><<<row_grid(a.rows), kLnThreads, 0, s>>>(dy, a.lddy, in, a.rows, a.cols, a.gamma, a.mean, a.rstd,
                                                             static_cast<const T*>(a.add), a.ldadd,
                                                             static_cast<T*>(a.dx), a.lddx);
    const unsigned ygrid = (unsigned)(chunks < 65535 ? chunks : 65535);
    k_ln_param_part<T><<<dim3(cgrid, ygrid), kLnThreads, 0, s>>>(dy, a.lddy, in, a.rows, a.cols, a.mean, a.rstd, a.part);
  }
  if (a.grad_dtype == ONEBIT_F32)
    k_ln_param_sum<<<cgrid, kLnThreads, 0, s>>>(a.part, chunks, a.cols, static_cast<float*>(a.dgamma), static_cast<float*>(a.dbeta));
  else if (a.grad_dtype == ONEBIT_F16)
    k_ln_param_sum<<<cgrid, kLnThreads, 0, s>>>(a.part, chunks, a.cols, static_cast<__half*>(a.dgamma), static_cast<__half*>(a.dbeta));
  else
    k_ln_param_sum<<<cgrid, kLnThreads, 0, s>>>(a.part, chunks, a.cols, static_cast<__nv_bfloat16*>(a.dgamma), static_cast<__nv_bfloat16*>(a.dbeta));
  return cudaGetLastError();
}

onebit_status_t shape_ok(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 1) return fail(ONEBIT_ERR_INVALID_ARG, "rows or columns out of range");
  if (rows > kMaxRows || cols > kMaxCols) return fail(ONEBIT_ERR_UNSUPPORTED, "more than 2^31 rows or 2^24 columns");
  return ONEBIT_OK;
}

}  // namespace
}  // namespace layers
}  // namespace onebit

using namespace onebit::layers;

extern "C" onebit_status_t onebit_layer_norm_forward(const void* x, int64_t ldx, int32_t dtype, int64_t rows,
                                                     int64_t cols, const float* gamma, const float* beta, float eps,
                                                     void* y, int64_t ldy, float* mean, float* rstd, int8_t* codes,
                                                     float* scales, onebit_stream_t stream) {
  onebit_status_t st = shape_ok(rows, cols);
  if (st != ONEBIT_OK) return st;
  if (!dtype_ok(dtype)) return fail(ONEBIT_ERR_INVALID_ARG, "dtype is not one of f32, f16, bf16");
  if (ldx < cols || ldy < cols) return fail(ONEBIT_ERR_INVALID_ARG, "a row stride below the columns");
  if (!(eps >= 0.0f)) return fail(ONEBIT_ERR_INVALID_ARG, "eps is negative or NaN");
  if (!codes != !scales) return fail(ONEBIT_ERR_INVALID_ARG, "a checkpoint needs codes and scales");
  if (rows == 0) return ONEBIT_OK;
  if (!x || !gamma || !beta || !y || !mean || !rstd) return fail(ONEBIT_ERR_INVALID_ARG, "a NULL buffer");
  const int64_t blocks = ceil_div(cols, kBlock), e = dtype_size(dtype);
  if (!aligned(x, e) || !aligned(y, e) || !aligned(gamma, 4) || !aligned(beta, 4) || !aligned(mean, 4) || !aligned(rstd, 4) ||
      !aligned(scales, 4))
    return fail(ONEBIT_ERR_INVALID_ARG, "a buffer is not aligned to its type");
  if (!disjoint({matrix(x, rows, ldx, cols, e), span_of(gamma, cols * 4), span_of(beta, cols * 4)},
                {matrix(y, rows, ldy, cols, e), span_of(mean, rows * 4), span_of(rstd, rows * 4),
                 span_of(codes, rows * cols), span_of(scales, rows * blocks * 4)}))
    return fail(ONEBIT_ERR_INVALID_ARG, "an output overlaps another buffer");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int grid = row_grid(rows);
  auto go = [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    k_ln_forward<T><<<grid, kLnThreads, 0, s>>>(static_cast<const T*>(x), ldx, rows, (int)cols, gamma, beta, eps,
                                                static_cast<T*>(y), ldy, mean, rstd, codes, scales, (int)blocks);
  };
  if (dtype == ONEBIT_F32) go((float*)nullptr);
  else if (dtype == ONEBIT_F16) go((__half*)nullptr);
  else go((__nv_bfloat16*)nullptr);
  const cudaError_t ce = cudaGetLastError();
  return ce == cudaSuccess ? ONEBIT_OK : cuda_fail(ce, "onebit_layer_norm_forward");
}

extern "C" onebit_status_t onebit_layer_norm_backward_workspace(int64_t rows, int64_t cols, size_t* bytes) {
  if (!bytes) return fail(ONEBIT_ERR_INVALID_ARG, "bytes is NULL");
  onebit_status_t st = shape_ok(rows, cols);
  if (st != ONEBIT_OK) return st;
  *bytes = (size_t)(ceil_div(rows, kRun) * 2 * cols * 4);
  return ONEBIT_OK;
}

extern "C" onebit_status_t onebit_layer_norm_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                                                      const int8_t* codes, const float* scales, int32_t dtype,
                                                      int64_t rows, int64_t cols, const float* gamma,
                                                      const float* mean, const float* rstd, const void* add,
                                                      int64_t ldadd, void* dx, int64_t lddx, void* dgamma,
                                                      void* dbeta, int32_t grad_dtype, void* workspace,
                                                      size_t workspace_bytes, onebit_stream_t stream) {
  size_t need = 0;
  onebit_status_t st = onebit_layer_norm_backward_workspace(rows, cols, &need);
  if (st != ONEBIT_OK) return st;
  if (!dtype_ok(dtype) || !dtype_ok(grad_dtype))
    return fail(ONEBIT_ERR_INVALID_ARG, "dtype is not one of f32, f16, bf16");
  if (!codes != !scales) return fail(ONEBIT_ERR_INVALID_ARG, "a checkpoint needs codes and scales");
  if (x && codes) return fail(ONEBIT_ERR_INVALID_ARG, "the input is x or its checkpoint, not both");
  if (lddy < cols || lddx < cols || (x && ldx < cols) || (add && ldadd < cols))
    return fail(ONEBIT_ERR_INVALID_ARG, "a row stride below the columns");
  if (!dgamma || !dbeta) return fail(ONEBIT_ERR_INVALID_ARG, "a NULL buffer");
  if (rows > 0 && (!dy || (!x && !codes) || !gamma || !mean || !rstd || !dx))
    return fail(ONEBIT_ERR_INVALID_ARG, "a NULL buffer");
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 16)))
    return fail(ONEBIT_ERR_WORKSPACE, "the workspace is too small or not 16-byte aligned");
  const int64_t blocks = ceil_div(cols, kBlock), e = dtype_size(dtype), ge = dtype_size(grad_dtype);
  if (!aligned(dy, e) || !aligned(x, e) || !aligned(add, e) || !aligned(dx, e) || !aligned(scales, 4) || !aligned(gamma, 4) ||
      !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(dgamma, ge) || !aligned(dbeta, ge))
    return fail(ONEBIT_ERR_INVALID_ARG, "a buffer is not aligned to its type");
  if (!disjoint({matrix(dy, rows, lddy, cols, e), matrix(x, rows, ldx, cols, e), span_of(codes, rows * cols),
                 span_of(scales, rows * blocks * 4), span_of(gamma, cols * 4), span_of(mean, rows * 4),
                 span_of(rstd, rows * 4), matrix(add, rows, ldadd, cols, e)},
                {matrix(dx, rows, lddx, cols, e), span_of(dgamma, cols * ge), span_of(dbeta, cols * ge),
                 span_of(workspace, (int64_t)need)}))
    return fail(ONEBIT_ERR_INVALID_ARG, "an output overlaps another buffer");
  const BackwardArgs a{dy, lddy, x, ldx, codes, scales, rows, (int)cols, (int)blocks, gamma, mean, rstd, add, ldadd,
                       dx, lddx, dgamma, dbeta, grad_dtype, static_cast<float*>(workspace)};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t ce = dtype == ONEBIT_F32 ? launch_backward<float>(a, s)
                         : dtype == ONEBIT_F16 ? launch_backward<__half>(a, s)
                                               : launch_backward<__nv_bfloat16>(a, s);
  return ce == cudaSuccess ? ONEBIT_OK : cuda_fail(ce, "onebit_layer_norm_backward");
}
