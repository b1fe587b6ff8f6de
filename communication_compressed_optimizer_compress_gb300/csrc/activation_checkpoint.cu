// activation_checkpoint.cu -- activations held in 8 bits: int8 codes with one fp32 scale per 64
// columns of a row.  See include/onebit_layers.h for the formulas.
#include <stdio.h>

#include <string>

#include "layers_common.cuh"

namespace onebit {
namespace layers {

namespace {
thread_local std::string t_error;
}  // namespace

onebit_status_t fail(onebit_status_t status, const char* what) {
  try {
    t_error = what;
  } catch (...) {  // out of memory for the message: no exception crosses the C boundary
    t_error.clear();
  }
  return status;
}
onebit_status_t cuda_fail(cudaError_t e, const char* where) {
  char buf[256];
  snprintf(buf, sizeof buf, "%s: %s", where, cudaGetErrorString(e));
  return fail(ONEBIT_ERR_CUDA, buf);
}
const char* error_text() { return t_error.c_str(); }

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
      n < 1)
    return 1;
  return n;
}

namespace {

constexpr int kCkThreads = 256;

// One warp per block of 64 columns of a row; a lane holds columns lane and lane + 32 of it.
template <typename T>
__global__ void __launch_bounds__(kCkThreads) k_compress(const T* __restrict__ x, int64_t ldx, int64_t rows, int cols,
                                                         int blocks, int8_t* __restrict__ codes,
                                                         float* __restrict__ scales) {
  const int lane = threadIdx.x & 31;
  const int64_t units = rows * blocks, step = (int64_t)gridDim.x * (kCkThreads / 32);
  for (int64_t u = (int64_t)blockIdx.x * (kCkThreads / 32) + (threadIdx.x >> 5); u < units; u += step) {
    const int64_t r = u / blocks;
    const int c0 = (int)(u - r * blocks) * kBlock + lane, c1 = c0 + 32;
    const float v0 = c0 < cols ? to_f(x[r * ldx + c0]) : 0.0f;
    const float v1 = c1 < cols ? to_f(x[r * ldx + c1]) : 0.0f;
    const BlockScale s = block_scale(warp_max_nan(max_nan(fabsf(v0), fabsf(v1))));
    if (c0 < cols) codes[r * cols + c0] = (int8_t)code_of(v0, s.inv);
    if (c1 < cols) codes[r * cols + c1] = (int8_t)code_of(v1, s.inv);
    if (lane == 0) scales[u] = s.scale;
  }
}

template <typename T>
__global__ void __launch_bounds__(kCkThreads) k_restore(const int8_t* __restrict__ codes,
                                                        const float* __restrict__ scales, int64_t rows, int cols,
                                                        int blocks, int act, T* __restrict__ x, int64_t ldx) {
  const int lane = threadIdx.x & 31;
  const int64_t units = rows * blocks, step = (int64_t)gridDim.x * (kCkThreads / 32);
  for (int64_t u = (int64_t)blockIdx.x * (kCkThreads / 32) + (threadIdx.x >> 5); u < units; u += step) {
    const int64_t r = u / blocks;
    const float s = scales[u];
    for (int c = (int)(u - r * blocks) * kBlock + lane, k = 0; k < 2 && c < cols; ++k, c += 32)
      x[r * ldx + c] = from_f<T>(act_value(act, value_of<T>(codes[r * cols + c], s)));
  }
}

int ck_grid(int64_t units) {
  const int64_t most = (int64_t)sm_count() * 8, want = ceil_div(units, kCkThreads / 32);
  return (int)(want < most ? want : most);
}

}  // namespace
}  // namespace layers
}  // namespace onebit

using namespace onebit::layers;

extern "C" const char* onebit_layers_last_error(void) { return onebit::layers::error_text(); }

static onebit_status_t checkpoint_args(const void* x, int64_t ldx, int32_t dtype, int64_t rows, int64_t cols,
                                       const int8_t* codes, const float* scales) {
  if (!dtype_ok(dtype)) return fail(ONEBIT_ERR_INVALID_ARG, "dtype is not one of f32, f16, bf16");
  if (rows < 0 || cols < 1 || ldx < cols) return fail(ONEBIT_ERR_INVALID_ARG, "rows, columns or row stride out of range");
  if (rows > kMaxRows || cols > kMaxCols) return fail(ONEBIT_ERR_UNSUPPORTED, "more than 2^31 rows or 2^24 columns");
  if (rows > 0 && (!x || !codes || !scales)) return fail(ONEBIT_ERR_INVALID_ARG, "a NULL buffer");
  if (!aligned(x, dtype_size(dtype)) || !aligned(scales, 4))
    return fail(ONEBIT_ERR_INVALID_ARG, "a buffer is not aligned to its type");
  return ONEBIT_OK;
}

extern "C" onebit_status_t onebit_checkpoint_compress(const void* x, int64_t ldx, int32_t dtype, int64_t rows,
                                                      int64_t cols, int8_t* codes, float* scales,
                                                      onebit_stream_t stream) {
  onebit_status_t st = checkpoint_args(x, ldx, dtype, rows, cols, codes, scales);
  if (st != ONEBIT_OK || rows == 0) return st;
  const int64_t blocks = ceil_div(cols, kBlock);
  if (!disjoint({matrix(x, rows, ldx, cols, dtype_size(dtype))}, {span_of(codes, rows * cols), span_of(scales, rows * blocks * 4)}))
    return fail(ONEBIT_ERR_INVALID_ARG, "an output overlaps another buffer");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int grid = ck_grid(rows * blocks);
  if (dtype == ONEBIT_F32)
    k_compress<<<grid, kCkThreads, 0, s>>>(static_cast<const float*>(x), ldx, rows, (int)cols, (int)blocks, codes, scales);
  else if (dtype == ONEBIT_F16)
    k_compress<<<grid, kCkThreads, 0, s>>>(static_cast<const __half*>(x), ldx, rows, (int)cols, (int)blocks, codes, scales);
  else
    k_compress<<<grid, kCkThreads, 0, s>>>(static_cast<const __nv_bfloat16*>(x), ldx, rows, (int)cols, (int)blocks, codes, scales);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? ONEBIT_OK : cuda_fail(e, "onebit_checkpoint_compress");
}

extern "C" onebit_status_t onebit_checkpoint_restore(const int8_t* codes, const float* scales, int64_t rows,
                                                     int64_t cols, int32_t activation, void* x, int64_t ldx,
                                                     int32_t dtype, onebit_stream_t stream) {
  onebit_status_t st = checkpoint_args(x, ldx, dtype, rows, cols, codes, scales);
  if (st != ONEBIT_OK) return st;
  if (activation < ONEBIT_ACT_NONE || activation > ONEBIT_ACT_GELU_TANH)
    return fail(ONEBIT_ERR_INVALID_ARG, "unknown activation");
  if (rows == 0) return ONEBIT_OK;
  const int64_t blocks = ceil_div(cols, kBlock);
  if (!disjoint({span_of(codes, rows * cols), span_of(scales, rows * blocks * 4)}, {matrix(x, rows, ldx, cols, dtype_size(dtype))}))
    return fail(ONEBIT_ERR_INVALID_ARG, "the output overlaps an input");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int grid = ck_grid(rows * blocks);
  if (dtype == ONEBIT_F32)
    k_restore<<<grid, kCkThreads, 0, s>>>(codes, scales, rows, (int)cols, (int)blocks, activation, static_cast<float*>(x), ldx);
  else if (dtype == ONEBIT_F16)
    k_restore<<<grid, kCkThreads, 0, s>>>(codes, scales, rows, (int)cols, (int)blocks, activation, static_cast<__half*>(x), ldx);
  else
    k_restore<<<grid, kCkThreads, 0, s>>>(codes, scales, rows, (int)cols, (int)blocks, activation, static_cast<__nv_bfloat16*>(x), ldx);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? ONEBIT_OK : cuda_fail(e, "onebit_checkpoint_restore");
}
