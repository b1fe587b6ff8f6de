// dropout.cu -- dropout of a matrix from a counter-based generator.  See include/onebit_layers.h for the definition.
#include <algorithm>

#include "unaligned.cuh"

namespace onebit {
namespace layers {
namespace {

// Blocks an SM.  Of dense rows as many as are there at once: more wait for the first to end, and then the SM is half empty (16384 x 4096
// bf16 49.9 us with eight of which six fit, 42.8 with six).  Odd rows are uneven work, and more blocks even it out (16384 x 1001 bf16 29.2 us
// with eight, 30.4 with six, 30.5 with four).
constexpr int kDenseBlocks = 6, kRowBlocks = 8;

// Dense rows on 32 bytes, of whole groups: a thread has 16 columns, two groups, at a time, whatever row they are in.  Bound by
// DRAM (94% of the copy rate; as long without dropout, so that the generator's instructions are hidden).
template <typename T>
__global__ void __launch_bounds__(256, kDenseBlocks) k_dropout_dense(const T* __restrict__ x, int64_t pairs, const Dropout d, T* __restrict__ y) {
  in_turn();
  const Generator gen(d);
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < pairs; i += (int64_t)gridDim.x * 256) {
    f2 v[2][4];
    load16(x + i * 16, &v[0][0]);
    if (d.threshold) gen.apply8(2 * i, v[0]), gen.apply8(2 * i + 1, v[1]);
    store16(y + i * 16, &v[0][0]);
  }
}

// Rows of any layout: WIDTH lanes have WIDTH groups of a row at a time, so that odd rows' vectors are put together from neighbouring
// lanes' values.  Bound by the instructions of the shifts and the generator (65% of the issue slots, the ALU 59% in fp32 and 69% in 16 bits): 4099 x
// 1155 fp32 10.1 us (18.5 by single elements), 16384 x 1001 bf16 29.3 (45.4).
template <typename T, int WIDTH, bool VEC>
__global__ void __launch_bounds__(256) k_dropout_rows(const T* __restrict__ x, int64_t ldx, int64_t rows, int cols, const Dropout d, T* __restrict__ y,
                                                      int64_t ldy) {
  in_turn();
  const Generator gen(d);
  const int64_t groups = (cols + 7) / 8;
  const int parts = (int)((groups + WIDTH - 1) / WIDTH), lane = threadIdx.x % WIDTH;
  // part p of row r, and as far as all lanes together go at a step
  const int64_t first = ((int64_t)blockIdx.x * 256 + threadIdx.x) / WIDTH, all = (int64_t)gridDim.x * (256 / WIDTH), dr = all / parts;
  int64_t r = first / parts;
  int p = (int)(first - r * parts);
  const int dp = (int)(all - dr * parts);
  while (r < rows) {
    const int c = (p * WIDTH + lane) * 8;
    f2 v[4];
    load_columns<T, VEC>(x + r * ldx, c, cols, v);
    if (d.threshold) gen.apply8(r * groups + c / 8, v);
    store_columns<T, WIDTH, VEC>(y + r * ldy, c, cols, v);
    r += dr, p += dp;
    if (p >= parts) p -= parts, ++r;
  }
}

template <typename T>
cudaError_t run(const void* px, int64_t ldx, int64_t rows, int64_t cols, const Dropout& d, void* py, int64_t ldy, cudaStream_t s) {
  const T* x = static_cast<const T*>(px);
  T* y = static_cast<T*>(py);
  const int64_t total = rows * cols;
  auto grid = [&](int64_t threads, int per_sm) { return (unsigned)std::min(ceil_div(threads, 256), (int64_t)sm_count() * per_sm); };
  if (cols % 8 == 0 && total % 16 == 0 && aligned(x, 32) && aligned(y, 32) && (rows == 1 || (ldx == cols && ldy == cols)))
    return launch_after(k_dropout_dense<T>, grid(total / 16, kDenseBlocks), 256, s, x, total / 16, d, y);
  auto on16 = [](const void* p, int64_t ld) { return aligned(p, 16) && (ld * (int64_t)sizeof(T)) % 16 == 0; };
  const bool vec = cols % 8 == 0 && on16(x, ldx) && on16(y, ldy);
  const int64_t groups = ceil_div(cols, 8);
  auto go = [&](auto* kernel, int64_t width) {
    return launch_after(kernel, grid(rows * ceil_div(groups, width) * width, kRowBlocks), 256, s, x, ldx, rows, (int)cols, d, y, ldy);
  };
  if (groups <= 8) return vec ? go(k_dropout_rows<T, 8, true>, 8) : go(k_dropout_rows<T, 8, false>, 8);
  return vec ? go(k_dropout_rows<T, 32, true>, 32) : go(k_dropout_rows<T, 32, false>, 32);
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
