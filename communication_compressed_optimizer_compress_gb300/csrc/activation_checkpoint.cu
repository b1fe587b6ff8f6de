// activation_checkpoint.cu -- activations held in 8 bits: int8 codes with one fp32 scale per 64
// columns of a row.  See include/onebit_layers.h for the formulas.
#include <stdio.h>

#include <atomic>
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
// A call's errors are its launches' own results, so that one that earlier code has left pending is not taken for it; its
// own is not left pending for the next caller either.
onebit_status_t cuda_fail(cudaError_t e, const char* where) {
  cudaGetLastError();
  char buf[256];
  snprintf(buf, sizeof buf, "%s: %s", where, cudaGetErrorString(e));
  return fail(ONEBIT_ERR_CUDA, buf);
}
const char* error_text() { return t_error.c_str(); }

int sm_count() {
  static std::atomic<int> known[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 1;
  if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return 1;
  if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

namespace {

// Both kernels move every byte once and are bound by that.  Wide form: a thread has 16 columns (32 or 64
// bytes in, 16 bytes of codes out), so that four threads share a scale and find the block's largest
// magnitude with two shuffles; a block takes runs of about kCkRun elements of whole rows.  It needs rows
// that start on 32 bytes, codes on 16 and a multiple of 16 columns.  Any other matrix takes the narrow form: one warp
// per 64 columns, a lane with two of them.  16384 x 4096 bf16: 36 us each way back to back, 205 MB at 5.7 TB/s (83% of
// a plain copy's rate).
constexpr int kCkThreads = 256;
constexpr int kCkRun = 16384;

// Columns and rows of a run: unit u of a run is 16 columns of row u / (4 blocks).
struct Wide {
  int64_t rows;
  int cols, blocks, run_rows;
};

template <typename T>
__global__ void __launch_bounds__(kCkThreads) k_compress_wide(const T* __restrict__ x, int64_t ldx, Wide w, int8_t* __restrict__ codes,
                                                              float* __restrict__ scales) {
  in_turn();
  const int per = 4 * w.blocks;
  const int64_t runs = (w.rows + w.run_rows - 1) / w.run_rows;
  for (int64_t run = blockIdx.x; run < runs; run += gridDim.x) {
    const int64_t r0 = run * w.run_rows;
    const int rows = (int)(w.rows - r0 < w.run_rows ? w.rows - r0 : w.run_rows), units = rows * per;
    for (int u0 = 0; u0 < units; u0 += kCkThreads) {
      const int u = u0 + threadIdx.x, r = u / per, g = u - r * per;
      const bool on = u < units && g * 16 < w.cols;
      f2 v[8];
      float most = 0.0f;
      if (on) {
        const T* p = x + (r0 + r) * ldx + g * 16;
        load16(p, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) most = max_abs(most, v[i]);
      }
      most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, 1));
      most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, 2));
      if (on) {
        const BlockScale s = block_scale(most);
        uint32_t c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = codes4(v[2 * i], v[2 * i + 1], s.inv);
        *reinterpret_cast<uint4*>(codes + (r0 + r) * w.cols + g * 16) = make_uint4(c[0], c[1], c[2], c[3]);
        if ((g & 3) == 0) scales[(r0 + r) * w.blocks + g / 4] = s.scale;
      }
    }
  }
}

template <typename T, int ACT>
__global__ void __launch_bounds__(kCkThreads) k_restore_wide(const int8_t* __restrict__ codes, const float* __restrict__ scales, Wide w,
                                                             T* __restrict__ x, int64_t ldx) {
  in_turn();
  const int per = w.cols / 16;
  const ActConsts k = literal_consts<ACT>();
  const int64_t runs = (w.rows + w.run_rows - 1) / w.run_rows;
  for (int64_t run = blockIdx.x; run < runs; run += gridDim.x) {
    const int64_t r0 = run * w.run_rows;
    const int rows = (int)(w.rows - r0 < w.run_rows ? w.rows - r0 : w.run_rows), units = rows * per;
#pragma unroll 2
    for (int u = threadIdx.x; u < units; u += kCkThreads) {
      const int r = u / per, g = u - r * per;
      const uint4 c = __ldg(reinterpret_cast<const uint4*>(codes + (r0 + r) * w.cols + g * 16));
      const float s = __ldg(scales + (r0 + r) * w.blocks + g / 4);
      f2 v[8];
      values4<T>(c.x, s, v), values4<T>(c.y, s, v + 2), values4<T>(c.z, s, v + 4), values4<T>(c.w, s, v + 6);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = act2<ACT>(k, v[i]);
      T* p = x + (r0 + r) * ldx + g * 16;
      store16(p, v);
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kCkThreads) k_compress(const T* __restrict__ x, int64_t ldx, int64_t rows, int cols,
                                                         int blocks, int8_t* __restrict__ codes,
                                                         float* __restrict__ scales) {
  in_turn();
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
  in_turn();
  const int lane = threadIdx.x & 31;
  const int64_t units = rows * blocks, step = (int64_t)gridDim.x * (kCkThreads / 32);
  for (int64_t u = (int64_t)blockIdx.x * (kCkThreads / 32) + (threadIdx.x >> 5); u < units; u += step) {
    const int64_t r = u / blocks;
    const float s = scales[u];
    for (int c = (int)(u - r * blocks) * kBlock + lane, k = 0; k < 2 && c < cols; ++k, c += 32)
      x[r * ldx + c] = from_f<T>(act_value(act, value_of<T>(codes[r * cols + c], s)));
  }
}

bool wide_ok(const void* x, int64_t ldx, int32_t dtype, int64_t cols, const int8_t* codes) {
  return aligned(x, 32) && (ldx * dtype_size(dtype)) % 32 == 0 && cols % 16 == 0 && aligned(codes, 16);
}
unsigned ck_grid(int64_t units) {
  const int64_t most = (int64_t)sm_count() * 8;
  return (unsigned)(units < most ? units : most);
}

template <typename T>
cudaError_t compress(const void* x, int64_t ldx, int32_t dtype, int64_t rows, int cols, int8_t* codes, float* scales, cudaStream_t s) {
  const int blocks = (int)ceil_div(cols, kBlock);
  const T* p = static_cast<const T*>(x);
  if (wide_ok(x, ldx, dtype, cols, codes)) {
    const Wide w{rows, cols, blocks, cols < kCkRun ? kCkRun / cols : 1};
    return launch_after(k_compress_wide<T>, ck_grid(ceil_div(rows, w.run_rows)), kCkThreads, s, p, ldx, w, codes, scales);
  }
  return launch_after(k_compress<T>, ck_grid(ceil_div(rows * blocks, kCkThreads / 32)), kCkThreads, s, p, ldx, rows, cols, blocks, codes, scales);
}
template <typename T>
cudaError_t restore(const int8_t* codes, const float* scales, int64_t rows, int cols, int act, void* x, int64_t ldx, int32_t dtype, cudaStream_t s) {
  const int blocks = (int)ceil_div(cols, kBlock);
  T* p = static_cast<T*>(x);
  if (wide_ok(x, ldx, dtype, cols, codes)) {
    const Wide w{rows, cols, blocks, cols < kCkRun ? kCkRun / cols : 1};
    const unsigned grid = ck_grid(ceil_div(rows, w.run_rows));
    if (act == ONEBIT_ACT_NONE) return launch_after(k_restore_wide<T, ONEBIT_ACT_NONE>, grid, kCkThreads, s, codes, scales, w, p, ldx);
    if (act == ONEBIT_ACT_RELU) return launch_after(k_restore_wide<T, ONEBIT_ACT_RELU>, grid, kCkThreads, s, codes, scales, w, p, ldx);
    if (act == ONEBIT_ACT_GELU) return launch_after(k_restore_wide<T, ONEBIT_ACT_GELU>, grid, kCkThreads, s, codes, scales, w, p, ldx);
    return launch_after(k_restore_wide<T, ONEBIT_ACT_GELU_TANH>, grid, kCkThreads, s, codes, scales, w, p, ldx);
  }
  return launch_after(k_restore<T>, ck_grid(ceil_div(rows * blocks, kCkThreads / 32)), kCkThreads, s, codes, scales, rows, cols, blocks, act, p, ldx);
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
  const cudaError_t e = dtype == ONEBIT_F32   ? compress<float>(x, ldx, dtype, rows, (int)cols, codes, scales, s)
                        : dtype == ONEBIT_F16 ? compress<__half>(x, ldx, dtype, rows, (int)cols, codes, scales, s)
                                              : compress<__nv_bfloat16>(x, ldx, dtype, rows, (int)cols, codes, scales, s);
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
  const cudaError_t e = dtype == ONEBIT_F32   ? restore<float>(codes, scales, rows, (int)cols, activation, x, ldx, dtype, s)
                        : dtype == ONEBIT_F16 ? restore<__half>(codes, scales, rows, (int)cols, activation, x, ldx, dtype, s)
                                              : restore<__nv_bfloat16>(codes, scales, rows, (int)cols, activation, x, ldx, dtype, s);
  return e == cudaSuccess ? ONEBIT_OK : cuda_fail(e, "onebit_checkpoint_restore");
}
