// linear.cu -- the linear layer: matrix product with bias, activation, residual and an 8-bit checkpoint
// in its epilogue, and its backward pass.  See include/onebit_layers.h for the formulas.
#include "layers_common.cuh"

namespace onebit {
namespace layers {
namespace {

// ------------------------------------------------------------------------------------------------
// C[m][n] = sum_k A(m,k) B(n,k) in fp32.  A(m,k) is at a + m*am + k*ak, B(n,k) at b + n*bn + k*bk.
// Every kFold terms the running sum is added to the total, so that a long sum (600000 tokens) loses no
// more than a short one.
constexpr int kT = 64, kTK = 16, kFold = 1024;

template <typename T>
__global__ void __launch_bounds__(256) k_product(const T* __restrict__ a, int64_t am, int64_t ak,
                                                 const T* __restrict__ b, int64_t bn, int64_t bk, int64_t m, int64_t n,
                                                 int64_t k, float* __restrict__ c) {
  __shared__ float sa[kTK][kT + 4], sb[kTK][kT + 4];
  const int64_t ntiles = (n + kT - 1) / kT, tiles = (m + kT - 1) / kT * ntiles;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t m0 = tile / ntiles * kT, n0 = tile % ntiles * kT;
    float acc[4][4] = {}, total[4][4] = {};
    for (int64_t k0 = 0; k0 < k; k0 += kTK) {
      __syncthreads();
      for (int q = threadIdx.x; q < kT * kTK; q += 256) {
        // walk along whichever index is contiguous in memory
        const int am_ = ak == 1 ? q / kTK : q % kT, ak_ = ak == 1 ? q % kTK : q / kT;
        sa[ak_][am_] = m0 + am_ < m && k0 + ak_ < k ? to_f(a[(m0 + am_) * am + (k0 + ak_) * ak]) : 0.0f;
        const int bn_ = bk == 1 ? q / kTK : q % kT, bk_ = bk == 1 ? q % kTK : q / kT;
        sb[bk_][bn_] = n0 + bn_ < n && k0 + bk_ < k ? to_f(b[(n0 + bn_) * bn + (k0 + bk_) * bk]) : 0.0f;
      }
      __syncthreads();
#pragma unroll
      for (int q = 0; q < kTK; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[q][ty * 4 + i], sb[q][tx * 4 + j], acc[i][j]);
      if ((k0 + kTK) % kFold == 0 || k0 + kTK >= k) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            total[i][j] += acc[i][j];
            acc[i][j] = 0.0f;
          }
      }
    }
    for (int i = 0; i < 4; ++i)
      for (int j = 0; j < 4; ++j)
        if (m0 + ty * 4 + i < m && n0 + tx * 4 + j < n) c[(m0 + ty * 4 + i) * n + n0 + tx * 4 + j] = total[i][j];
  }
}

// ------------------------------------------------------------------------------------------------
// Epilogues over the fp32 product, one warp per 64 columns of a row.

template <typename T>
struct ForwardEpilogue {
  const float* bias;
  const T* residual;
  int64_t ldr;
  T* y;
  int64_t ldy;
  int8_t* codes;
  float* scales;
  int act;
};

template <typename T>
__global__ void __launch_bounds__(256) k_finish_forward(const float* __restrict__ c, int64_t rows, int cols, int blocks,
                                                        ForwardEpilogue<T> e) {
  const int lane = threadIdx.x & 31;
  const int64_t units = rows * blocks, step = (int64_t)gridDim.x * 8;
  for (int64_t u = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); u < units; u += step) {
    const int64_t r = u / blocks;
    const int c0 = (int)(u - r * blocks) * kBlock + lane;
    float z[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int col = c0 + 32 * q;
      z[q] = 0.0f;
      if (col < cols) {
        z[q] = c[r * cols + col] + (e.bias ? e.bias[col] : 0.0f);
        float v = act_value(e.act, z[q]);
        if (e.residual) v += to_f(e.residual[r * e.ldr + col]);
        e.y[r * e.ldy + col] = from_f<T>(v);
      }
    }
    if (e.codes) {
      const BlockScale s = block_scale(warp_max_nan(max_nan(fabsf(z[0]), fabsf(z[1]))));
#pragma unroll
      for (int q = 0; q < 2; ++q)
        if (c0 + 32 * q < cols) e.codes[r * cols + c0 + 32 * q] = (int8_t)code_of(z[q], s.inv);
      if (lane == 0) e.scales[u] = s.scale;
    }
  }
}

// The value before the activation as the backward pass has it: itself, or its 8-bit checkpoint.
template <typename T>
struct Kept {
  const T* x;
  int64_t ldx;
  const int8_t* codes;
  const float* scales;
  int cols, blocks;
  __device__ __forceinline__ float at(int64_t r, int c) const {
    return codes ? value_of<T>(codes[r * cols + c], scales[r * blocks + c / kBlock]) : to_f(x[r * ldx + c]);
  }
};

// dx = c * act'(v) [+ add]
template <typename T>
__global__ void __launch_bounds__(256) k_finish_dx(const float* __restrict__ c, int64_t rows, int cols, Kept<T> v, int act,
                                                   const T* __restrict__ add, int64_t ldadd, T* __restrict__ dx,
                                                   int64_t lddx) {
  const int64_t total = rows * cols;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / cols;
    const int col = (int)(i - r * cols);
    float d = c[i];
    if (act != ONEBIT_ACT_NONE) d *= act_slope(act, v.at(r, col));
    if (add) d += to_f(add[r * ldadd + col]);
    dx[r * lddx + col] = from_f<T>(d);
  }
}

// h = act(v), rounded to the product's operand type
template <typename T>
__global__ void __launch_bounds__(256) k_operand(Kept<T> v, int64_t rows, int cols, int act, T* __restrict__ h) {
  const int64_t total = rows * cols;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / cols;
    h[i] = from_f<T>(act_value(act, v.at(r, (int)(i - r * cols))));
  }
}

template <typename G>
__global__ void __launch_bounds__(256) k_round(const float* __restrict__ c, int64_t total, G* __restrict__ out) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) out[i] = from_f<G>(c[i]);
}

// Column sums: part[chunk][cols] over runs of kRun rows, then their sum in chunk order.
constexpr int kRun = 128;
template <typename T>
__global__ void __launch_bounds__(256) k_colsum_part(const T* __restrict__ dy, int64_t lddy, int64_t rows, int cols,
                                                     float* __restrict__ part) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= cols) return;
  for (int64_t ch = blockIdx.y; ch * kRun < rows; ch += gridDim.y) {
    const int64_t end = (ch + 1) * kRun < rows ? (ch + 1) * kRun : rows;
    float b = 0.0f;
    for (int64_t r = ch * kRun; r < end; ++r) b += to_f(dy[r * lddy + c]);
    part[ch * cols + c] = b;
  }
}
template <typename G>
__global__ void __launch_bounds__(256) k_colsum_sum(const float* __restrict__ part, int64_t chunks, int cols,
                                                    G* __restrict__ db) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= cols) return;
  float b = 0.0f;
  for (int64_t ch = 0; ch < chunks; ++ch) b += part[ch * cols + c];
  db[c] = from_f<G>(b);
}

int flat_grid(int64_t total) {
  const int64_t most = (int64_t)sm_count() * 8, want = ceil_div(total, 256);
  return (int)(want < most ? want : most);
}

template <typename T>
void product(const T* a, int64_t am, int64_t ak, const T* b, int64_t bn, int64_t bk, int64_t m, int64_t n, int64_t k,
             float* c, cudaStream_t s) {
  const int64_t tiles = ceil_div(m, kT) * ceil_div(n, kT), most = (int64_t)sm_count() * 8;
  k_product<T><<<(unsigned)(tiles < most ? tiles : most), 256, 0, s>>>(a, am, ak, b, bn, bk, m, n, k, c);
}

// fp32 results of a type the caller names
template <typename F>
void with_grad(int32_t dtype, void* p, F&& f) {
  if (dtype == ONEBIT_F32) f(static_cast<float*>(p));
  else if (dtype == ONEBIT_F16) f(static_cast<__half*>(p));
  else f(static_cast<__nv_bfloat16*>(p));
}

int64_t pad256(int64_t b) { return (b + 255) & ~(int64_t)255; }

template <typename T>
cudaError_t forward(const onebit_linear_t& a, float* c, cudaStream_t s) {
  product<T>(static_cast<const T*>(a.x), a.ldx, 1, static_cast<const T*>(a.w), a.ldw, 1, a.rows, a.out, a.in, c, s);
  const int blocks = (int)ceil_div(a.out, kBlock);
  const ForwardEpilogue<T> e{a.bias, static_cast<const T*>(a.residual), a.ldr, static_cast<T*>(a.y), a.ldy, a.codes, a.scales, a.activation};
  k_finish_forward<T><<<flat_grid(a.rows * blocks * 32), 256, 0, s>>>(c, a.rows, (int)a.out, blocks, e);
  return cudaGetLastError();
}

// Workspace of the backward pass: the fp32 product (dx's or dw's), the operand act(v), db's partials.
struct BackwardSpace {
  int64_t product, operand, part;
  bool copies;  // act(v) has to be computed
  int64_t total() const { return product + operand + part; }
};
BackwardSpace backward_space(const onebit_linear_grad_t& a) {
  BackwardSpace b{};
  b.copies = a.dw && (a.codes || a.activation != ONEBIT_ACT_NONE);
  const int64_t p = a.dx ? a.rows * a.in * 4 : 0, q = a.dw ? a.out * a.in * 4 : 0;
  b.product = pad256(p > q ? p : q);
  b.operand = b.copies ? pad256(a.rows * a.in * dtype_size(a.dtype)) : 0;
  b.part = a.db ? pad256(ceil_div(a.rows, kRun) * a.out * 4) : 0;
  return b;
}

template <typename T>
cudaError_t backward(const onebit_linear_grad_t& a, char* ws, cudaStream_t s) {
  const BackwardSpace sp = backward_space(a);
  float* c = reinterpret_cast<float*>(ws);
  T* h = reinterpret_cast<T*>(ws + sp.product);
  float* part = reinterpret_cast<float*>(ws + sp.product + sp.operand);
  const T* dy = static_cast<const T*>(a.dy);
  const Kept<T> v{static_cast<const T*>(a.x), a.ldx, a.codes, a.scales, (int)a.in, (int)ceil_div(a.in, kBlock)};
  if (a.dx && a.rows > 0) {
    product<T>(dy, a.lddy, 1, static_cast<const T*>(a.w), 1, a.ldw, a.rows, a.in, a.out, c, s);
    k_finish_dx<T><<<flat_grid(a.rows * a.in), 256, 0, s>>>(c, a.rows, (int)a.in, v, a.activation, static_cast<const T*>(a.add), a.ldadd,
                                                            static_cast<T*>(a.dx), a.lddx);
  }
  if (a.dw) {
    const T* x = v.x;
    int64_t ldx = a.ldx;
    if (sp.copies && a.rows > 0) {
      k_operand<T><<<flat_grid(a.rows * a.in), 256, 0, s>>>(v, a.rows, (int)a.in, a.activation, h);
      x = h;
      ldx = a.in;
    }
    product<T>(dy, 1, a.lddy, x, 1, ldx, a.out, a.in, a.rows, c, s);
    with_grad(a.grad_dtype, a.dw, [&](auto* g) { k_round<<<flat_grid(a.out * a.in), 256, 0, s>>>(c, a.out * a.in, g); });
  }
  if (a.db) {
    const int64_t chunks = ceil_div(a.rows, kRun);
    const unsigned cgrid = (unsigned)ceil_div(a.out, 256);
    if (chunks)
      k_colsum_part<T><<<dim3(cgrid, (unsigned)(chunks < 65535 ? chunks : 65535)), 256, 0, s>>>(dy, a.lddy, a.rows, (int)a.out, part);
    with_grad(a.grad_dtype, a.db, [&](auto* g) { k_colsum_sum<<<cgrid, 256, 0, s>>>(part, chunks, (int)a.out, g); });
  }
  return cudaGetLastError();
}

onebit_status_t shape_ok(int64_t rows, int64_t in, int64_t out, int32_t dtype, int32_t act) {
  if (rows < 0 || in < 1 || out < 1) return fail(ONEBIT_ERR_INVALID_ARG, "rows or widths out of range");
  if (rows > kMaxRows || in > kMaxCols || out > kMaxCols)
    return fail(ONEBIT_ERR_UNSUPPORTED, "more than 2^31 rows or a width above 2^24");
  if (!dtype_ok(dtype)) return fail(ONEBIT_ERR_INVALID_ARG, "dtype is not one of f32, f16, bf16");
  if (dtype == ONEBIT_F32) return fail(ONEBIT_ERR_UNSUPPORTED, "the linear layer takes f16 or bf16 operands");
  if (act < ONEBIT_ACT_NONE || act > ONEBIT_ACT_GELU_TANH) return fail(ONEBIT_ERR_INVALID_ARG, "unknown activation");
  return ONEBIT_OK;
}

onebit_status_t forward_ok(const onebit_linear_t* a) {
  if (!a) return fail(ONEBIT_ERR_INVALID_ARG, "the arguments are NULL");
  onebit_status_t st = shape_ok(a->rows, a->in, a->out, a->dtype, a->activation);
  if (st != ONEBIT_OK) return st;
  if (a->ldx < a->in || a->ldw < a->in || a->ldy < a->out || (a->residual && a->ldr < a->out))
    return fail(ONEBIT_ERR_INVALID_ARG, "a row stride below the columns");
  if (!a->codes != !a->scales) return fail(ONEBIT_ERR_INVALID_ARG, "a checkpoint needs codes and scales");
  if (a->rows > 0 && (!a->x || !a->w || !a->y)) return fail(ONEBIT_ERR_INVALID_ARG, "a NULL buffer");
  if (!aligned(a->x, 2) || !aligned(a->w, 2) || !aligned(a->y, 2) || !aligned(a->residual, 2) || !aligned(a->bias, 4) ||
      !aligned(a->scales, 4))
    return fail(ONEBIT_ERR_INVALID_ARG, "a buffer is not aligned to its type");
  return ONEBIT_OK;
}

onebit_status_t backward_ok(const onebit_linear_grad_t* a) {
  if (!a) return fail(ONEBIT_ERR_INVALID_ARG, "the arguments are NULL");
  onebit_status_t st = shape_ok(a->rows, a->in, a->out, a->dtype, a->activation);
  if (st != ONEBIT_OK) return st;
  if (!dtype_ok(a->grad_dtype)) return fail(ONEBIT_ERR_INVALID_ARG, "grad_dtype is not one of f32, f16, bf16");
  if (!a->codes != !a->scales) return fail(ONEBIT_ERR_INVALID_ARG, "a checkpoint needs codes and scales");
  if (a->x && a->codes) return fail(ONEBIT_ERR_INVALID_ARG, "the input is x or its checkpoint, not both");
  if (a->lddy < a->out || (a->x && a->ldx < a->in) || (a->dx && (a->ldw < a->in || a->lddx < a->in || (a->add && a->ldadd < a->in))))
    return fail(ONEBIT_ERR_INVALID_ARG, "a row stride below the columns");
  if (a->rows > 0) {
    if ((a->dx || a->dw || a->db) && !a->dy) return fail(ONEBIT_ERR_INVALID_ARG, "a NULL buffer");
    if (a->dx && !a->w) return fail(ONEBIT_ERR_INVALID_ARG, "dx needs the weight");
    if ((a->dw || (a->dx && a->activation != ONEBIT_ACT_NONE)) && !a->x && !a->codes)
      return fail(ONEBIT_ERR_INVALID_ARG, "dw and the activation's derivative need x or its checkpoint");
  }
  const uintptr_t g = (uintptr_t)dtype_size(a->grad_dtype);
  if (!aligned(a->dy, 2) || !aligned(a->x, 2) || !aligned(a->w, 2) || !aligned(a->add, 2) || !aligned(a->dx, 2) ||
      !aligned(a->scales, 4) || !aligned(a->dw, g) || !aligned(a->db, g))
    return fail(ONEBIT_ERR_INVALID_ARG, "a buffer is not aligned to its type");
  return ONEBIT_OK;
}

}  // namespace
}  // namespace layers
}  // namespace onebit

using namespace onebit::layers;

extern "C" onebit_status_t onebit_linear_forward_workspace(const onebit_linear_t* a, size_t* bytes) {
  onebit_status_t st = forward_ok(a);
  if (st != ONEBIT_OK) return st;
  if (!bytes) return fail(ONEBIT_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = (size_t)pad256(a->rows * a->out * 4);
  return ONEBIT_OK;
}

extern "C" onebit_status_t onebit_linear_forward(const onebit_linear_t* a, void* workspace, size_t workspace_bytes,
                                                 onebit_stream_t stream) {
  size_t need = 0;
  onebit_status_t st = onebit_linear_forward_workspace(a, &need);
  if (st != ONEBIT_OK || a->rows == 0) return st;
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256)))
    return fail(ONEBIT_ERR_WORKSPACE, "the workspace is too small or not 256-byte aligned");
  const int64_t blocks = ceil_div(a->out, kBlock);
  if (!disjoint({matrix(a->x, a->rows, a->ldx, a->in, 2), matrix(a->w, a->out, a->ldw, a->in, 2),
                 span_of(a->bias, a->out * 4), matrix(a->residual, a->rows, a->ldr, a->out, 2)},
                {matrix(a->y, a->rows, a->ldy, a->out, 2), span_of(a->codes, a->rows * a->out),
                 span_of(a->scales, a->rows * blocks * 4), span_of(workspace, (int64_t)need)}))
    return fail(ONEBIT_ERR_INVALID_ARG, "an output overlaps another buffer");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  float* c = static_cast<float*>(workspace);
  const cudaError_t e = a->dtype == ONEBIT_F16 ? forward<__half>(*a, c, s) : forward<__nv_bfloat16>(*a, c, s);
  return e == cudaSuccess ? ONEBIT_OK : cuda_fail(e, "onebit_linear_forward");
}

extern "C" onebit_status_t onebit_linear_backward_workspace(const onebit_linear_grad_t* a, size_t* bytes) {
  onebit_status_t st = backward_ok(a);
  if (st != ONEBIT_OK) return st;
  if (!bytes) return fail(ONEBIT_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = (size_t)backward_space(*a).total();
  return ONEBIT_OK;
}

extern "C" onebit_status_t onebit_linear_backward(const onebit_linear_grad_t* a, void* workspace,
                                                  size_t workspace_bytes, onebit_stream_t stream) {
  size_t need = 0;
  onebit_status_t st = onebit_linear_backward_workspace(a, &need);
  if (st != ONEBIT_OK) return st;
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256)))
    return fail(ONEBIT_ERR_WORKSPACE, "the workspace is too small or not 256-byte aligned");
  const int64_t blocks = ceil_div(a->in, kBlock), g = dtype_size(a->grad_dtype);
  if (!disjoint({matrix(a->dy, a->rows, a->lddy, a->out, 2), matrix(a->x, a->rows, a->ldx, a->in, 2),
                 span_of(a->codes, a->rows * a->in), span_of(a->scales, a->rows * blocks * 4),
                 matrix(a->w, a->out, a->ldw, a->in, 2), matrix(a->add, a->rows, a->ldadd, a->in, 2)},
                {matrix(a->dx, a->rows, a->lddx, a->in, 2), span_of(a->dw, a->out * a->in * g),
                 span_of(a->db, a->out * g), span_of(workspace, (int64_t)need)}))
    return fail(ONEBIT_ERR_INVALID_ARG, "an output overlaps another buffer");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  const cudaError_t e = a->dtype == ONEBIT_F16 ? backward<__half>(*a, ws, s) : backward<__nv_bfloat16>(*a, ws, s);
  return e == cudaSuccess ? ONEBIT_OK : cuda_fail(e, "onebit_linear_backward");
}
