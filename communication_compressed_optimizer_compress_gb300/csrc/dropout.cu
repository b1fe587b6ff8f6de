// dropout.cu -- dropout of a matrix from a counter-based generator.  See include/onebit_layers.h for the definition.
#include "dropout.cuh"

namespace onebit {
namespace layers {
namespace {

// A thread has a group of eight columns at a time.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) k_dropout(const T* __restrict__ x, int64_t ldx, int64_t rows, int cols, const Dropout d, T* __restrict__ y,
                                                 int64_t ldy) {
  in_turn();
  const Generator gen(d);
  const int64_t groups = (cols + 7) / 8, total = rows * groups;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / groups;
    const int c = (int)(i - r * groups) * 8;
    f2 v[4];
    load_group<T, VEC>(x + r * ldx + c, cols - c, v);
    if (d.threshold) gen.apply8(i, v);
    store_group8<T, VEC>(y + r * ldy + c, cols - c, v);
  }
}

template <typename T>
cudaError_t run(const void* x, int64_t ldx, int64_t rows, int64_t cols, const Dropout& d, void* y, int64_t ldy, cudaStream_t s) {
  auto on16 = [](const void* p, int64_t ld) { return aligned(p, 16) && (ld * (int64_t)sizeof(T)) % 16 == 0; };
  const int64_t want = ceil_div(rows * ceil_div(cols, 8), 256), most = (int64_t)sm_count() * 8;
  auto go = [&](auto* kernel) {
    return launch_after(kernel, (unsigned)(want < most ? want : most), 256, s, static_cast<const T*>(x), ldx, rows, (int)cols, d, static_cast<T*>(y), ldy);
  };
  return cols % 8 == 0 && on16(x, ldx) && on16(y, ldy) ? go(k_dropout<T, true>) : go(k_dropout<T, false>);
}

}  // namespace
}  // namespace layers
}  // namespace onebit

using namespace onebit::layers;

extern "C" onebit_status_t onebit_dropout(const void* x, int64_t ldx, int32_t dtype, int64_t rows, int64_t cols, float p, const int64_t* key,
                                          uint32_t site, void* y, int64_t ldy, onebit_stream_t stream) {
  if (rows < 0 || cols < 1) return fail(ONEBIT_ERR_INVALID_ARG, "rows or columns out of range");
  if (rows > kMaxRows || cols > kMaxCols) return fail(ONEBIT_ERR_UNSUPPORTED, "more than 2^31 rows or 2^24 columns");
  if (!dtype_ok(dtype)) return fail(ONEBIT_ERR_INVALID_ARG, "dtype is not one of f32, f16, bf16");
  if (ldx < cols || ldy < cols) return fail(ONEBIT_ERR_INVALID_ARG, "a row stride below the columns");
  Dropout d{};
  const onebit_status_t st = make_dropout(&d, p, key, site);
  if (st != ONEBIT_OK) return st;
  if (rows == 0) return ONEBIT_OK;
  const int64_t e = dtype_size(dtype);
  if (!x || !y) return fail(ONEBIT_ERR_INVALID_ARG, "a NULL buffer");
  if (!aligned(x, e) || !aligned(y, e)) return fail(ONEBIT_ERR_INVALID_ARG, "a buffer is not aligned to its type");
  if (!disjoint({matrix(x, rows, ldx, cols, e), span_of(key, 16)}, {matrix(y, rows, ldy, cols, e)}))
    return fail(ONEBIT_ERR_INVALID_ARG, "an output overlaps another buffer");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t err = dtype == ONEBIT_F32   ? run<float>(x, ldx, rows, cols, d, y, ldy, s)
                          : dtype == ONEBIT_F16 ? run<__half>(x, ldx, rows, cols, d, y, ldy, s)
                                                : run<__nv_bfloat16>(x, ldx, rows, cols, d, y, ldy, s);
  return err == cudaSuccess ? ONEBIT_OK : cuda_fail(err, "onebit_dropout");
}
