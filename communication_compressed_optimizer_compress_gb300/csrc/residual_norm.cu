// residual_norm.cu -- the residual sum with the norms around it: a block's output through its norm, dropout and gate
// onto the residual stream, and the norm before the next block, forward and backward with the parameters' gradients.
// See include/onebit_layers.h for the formulas.
#include <type_traits>

#include "dropout.cuh"

namespace onebit {
namespace layers {
namespace {

struct ForwardArgs {
  const void* x;
  int64_t ldx;
  const void* block;  // NULL: s = x
  int64_t ldblock;
  const float *gamma, *beta, *block_gamma, *block_beta, *gate;
  Dropout drop;
  void* s;
  int64_t lds;
  void* y;
  int64_t ldy;
  float *mean, *rstd, *block_mean, *block_rstd;
  int64_t rows;
  int cols, groups;
  bool layer;
  float inv_cols, eps, scale;
};

struct BackwardArgs {
  const void* dy;
  int64_t lddy;
  const void* ds;
  int64_t ldds;
  const void* s;
  int64_t lds;
  const void* block;
  int64_t ldblock;
  const float *gamma, *block_gamma, *block_beta, *gate;
  Dropout drop;
  const float *mean, *rstd, *block_mean, *block_rstd;
  void* dx;
  int64_t lddx;
  void* dblock;
  int64_t lddblock;
  int64_t rows;
  int cols, groups;
  bool layer;
  float inv_cols, scale;
  float* part;  // the parameters' partial sums
  float* sums;  // (rows read again:) each row's two sums behind the norm before the next block
};

// ------------------------------------------------------------------------------------------------
// Rows of any width, read again for each step: one block a row, a thread eight columns at a time.
constexpr int kWideThreads = 256;
constexpr int kWideWarps = kWideThreads / 32;
template <int N>
__device__ __forceinline__ void block_sums(float (&v)[N], float (*red)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
  __syncthreads();  // red may still be read from the sums before
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) red[threadIdx.x >> 5][i] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = 0.0f;
#pragma unroll
    for (int w = 0; w < kWideWarps; ++w) v[i] += red[w][i];
  }
}
// (mean, rstd) of eight columns at a time from get(column, values), which gives 0 past the end
template <typename Get>
__device__ __forceinline__ float2 row_statistics(Get&& get, int cols, bool layer, float inv_cols, float eps, float (*red)[1]) {
  float v[1], mean = 0.0f;
  if (layer) {
    f2 t = 0;
    for (int c = threadIdx.x * 8; c < cols; c += kWideThreads * 8) {
      f2 f[4];
      get(c, f);
#pragma unroll
      for (int e = 0; e < 4; ++e) t = add2(t, f[e]);
    }
    v[0] = sum_of(t);
    block_sums(v, red);
    mean = v[0] * inv_cols;
  }
  f2 t = 0;
  for (int c = threadIdx.x * 8; c < cols; c += kWideThreads * 8) {
    f2 f[4];
    get(c, f);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const f2 d = add2(f[e], pair(c + 2 * e < cols ? -mean : 0.0f, c + 2 * e + 1 < cols ? -mean : 0.0f));
      t = fma2(d, d, t);
    }
  }
  v[0] = sum_of(t);
  block_sums(v, red);
  return make_float2(mean, halves(rsqrt_rounded(splat(fmaf(v[0], inv_cols, eps)))).x);
}

// a parameter's eight columns, `none` where there is no parameter
__device__ __forceinline__ void param8(const float* p, int c, int cols, float none, f2 (&f)[4]) {
  if (!p) {
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = splat(none);
  } else {
    load_group<float, false>(p + c, cols - c, f);
  }
}

template <typename T>
__global__ void __launch_bounds__(kWideThreads) k_rn_forward_wide(const ForwardArgs A) {
  in_turn();
  __shared__ float red[kWideWarps][1];
  const Generator gen(A.drop);
  for (int64_t r = blockIdx.x; r < A.rows; r += gridDim.x) {
    const T* x = static_cast<const T*>(A.x) + r * A.ldx;
    const T* b = static_cast<const T*>(A.block) + r * A.ldblock;
    float2 bst = make_float2(0.0f, 1.0f);
    auto block = [&](int c, f2(&f)[4]) { load_group<T, false>(b + c, A.cols - c, f); };
    if (A.block_gamma) {
      bst = row_statistics(block, A.cols, A.layer, A.inv_cols, A.eps, red);
      if (threadIdx.x == 0) {
        if (A.block_mean) A.block_mean[r] = bst.x;
        A.block_rstd[r] = bst.y;
      }
    }
    auto sum = [&](int c, f2(&f)[4]) {
      load_group<T, false>(x + c, A.cols - c, f);
      if (!A.block) return;
      f2 n[4], p[4], q[4];
      block(c, n);
      if (A.block_gamma) {
        param8(A.block_gamma, c, A.cols, 0.0f, p);
        param8(A.block_beta, c, A.cols, 0.0f, q);
#pragma unroll
        for (int e = 0; e < 4; ++e) n[e] = fma2(mul2(add2(n[e], splat(-bst.x)), splat(bst.y)), p[e], q[e]);
      }
      if (A.drop.threshold) gen.apply8(r * A.groups + c / 8, n);
      param8(A.gate, c, A.cols, 1.0f, p);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        f[e] = fma2(mul2(n[e], splat(A.scale)), p[e], f[e]);
        const float2 h = halves(f[e]);  // past the end there is no column (without a gate there is no parameter to be 0 there)
        f[e] = pair(c + 2 * e < A.cols ? h.x : 0.0f, c + 2 * e + 1 < A.cols ? h.y : 0.0f);
      }
    };
    float2 st = make_float2(0.0f, 1.0f);
    if (A.gamma) {
      st = row_statistics(sum, A.cols, A.layer, A.inv_cols, A.eps, red);
      if (threadIdx.x == 0) {
        if (A.mean) A.mean[r] = st.x;
        A.rstd[r] = st.y;
      }
    }
    for (int c = threadIdx.x * 8; c < A.cols; c += kWideThreads * 8) {
      f2 f[4], p[4], q[4];
      sum(c, f);
      if (A.block) store_group8<T, false>(static_cast<T*>(A.s) + r * A.lds + c, A.cols - c, f);
      if (A.gamma) {
        param8(A.gamma, c, A.cols, 0.0f, p);
        param8(A.beta, c, A.cols, 0.0f, q);
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = fma2(mul2(add2(f[e], splat(-st.x)), splat(st.y)), p[e], q[e]);
        store_group8<T, false>(static_cast<T*>(A.y) + r * A.ldy + c, A.cols - c, f);
      }
    }
  }
}

// What a row's columns pass on backward, eight of them: shat, dy and t, the gradient of s; d and n behind it.
template <typename T>
struct RowBackward {
  const BackwardArgs& A;
  const Generator& gen;
  int64_t r;
  float mean, rstd, block_mean, block_rstd;
  __device__ __forceinline__ RowBackward(const BackwardArgs& a, const Generator& g, int64_t row)
      : A(a), gen(g), r(row), mean(a.mean ? a.mean[row] : 0.0f), rstd(a.rstd ? a.rstd[row] : 0.0f), block_mean(a.block_mean ? a.block_mean[row] : 0.0f),
        block_rstd(a.block_rstd ? a.block_rstd[row] : 0.0f) {}
  __device__ __forceinline__ void load(const void* p, int64_t ld, int c, f2 (&f)[4]) const {
    load_group<T, false>(static_cast<const T*>(p) + r * ld + c, A.cols - c, f);
  }
  __device__ __forceinline__ void before(int c, f2 (&dy)[4], f2 (&shat)[4]) const {  // with gamma
    load(A.dy, A.lddy, c, dy);
    load(A.s, A.lds, c, shat);
#pragma unroll
    for (int e = 0; e < 4; ++e) shat[e] = mul2(add2(shat[e], splat(-mean)), splat(rstd));
  }
  // t, from the row's means of q and q shat
  __device__ __forceinline__ void t(int c, float m0, float m1, f2 (&out)[4]) const {
    f2 ds[4];
    if (A.ds) load(A.ds, A.ldds, c, ds);
    if (A.gamma) {
      f2 dy[4], shat[4], g[4];
      before(c, dy, shat);
      param8(A.gamma, c, A.cols, 0.0f, g);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        out[e] = mul2(fma2(shat[e], splat(-m1), fma2(dy[e], g[e], splat(-m0))), splat(rstd));
        if (A.ds) out[e] = add2(out[e], ds[e]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) out[e] = ds[e];
    }
  }
  // d = scale t mask, from t
  __device__ __forceinline__ void through(int c, f2 (&v)[4]) const {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = mul2(v[e], splat(A.scale));
    if (A.drop.threshold) gen.apply8(r * A.groups + c / 8, v);
  }
  __device__ __forceinline__ void bhat(int c, f2 (&b)[4]) const {  // normalised behind a norm, else the block itself
    load(A.block, A.ldblock, c, b);
    if (A.block_gamma) {
#pragma unroll
      for (int e = 0; e < 4; ++e) b[e] = mul2(add2(b[e], splat(-block_mean)), splat(block_rstd));
    }
  }
  // f = d gate block_gamma, from d; 0 past the end
  __device__ __forceinline__ void gated(int c, f2 (&v)[4]) const {
    f2 p[4], q[4];
    param8(A.gate, c, A.cols, 1.0f, p);
    param8(A.block_gamma, c, A.cols, 1.0f, q);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = mul2(mul2(v[e], p[e]), q[e]);
  }
};

template <typename T>
__global__ void __launch_bounds__(kWideThreads) k_rn_backward_wide(const BackwardArgs A) {
  in_turn();
  __shared__ float red[kWideWarps][2];
  const Generator gen(A.drop);
  for (int64_t r = blockIdx.x; r < A.rows; r += gridDim.x) {
    const RowBackward<T> row(A, gen, r);
    float m[2] = {0.0f, 0.0f};
    if (A.gamma) {
      f2 s0 = 0, s1 = 0;
      for (int c = threadIdx.x * 8; c < A.cols; c += kWideThreads * 8) {
        f2 dy[4], shat[4], g[4];
        row.before(c, dy, shat);
        param8(A.gamma, c, A.cols, 0.0f, g);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const f2 q = mul2(dy[e], g[e]);
          s0 = add2(s0, q);
          s1 = fma2(q, shat[e], s1);
        }
      }
      m[0] = sum_of(s0), m[1] = sum_of(s1);
      block_sums(m, red);
      m[0] = A.layer ? m[0] * A.inv_cols : 0.0f;
      m[1] *= A.inv_cols;
      if (threadIdx.x == 0) A.sums[2 * r] = m[0], A.sums[2 * r + 1] = m[1];
    }
    float n[2] = {0.0f, 0.0f};
    if (A.block_gamma) {
      f2 s0 = 0, s1 = 0;
      for (int c = threadIdx.x * 8; c < A.cols; c += kWideThreads * 8) {
        f2 v[4], b[4];
        row.t(c, m[0], m[1], v);
        row.through(c, v);
        row.gated(c, v);
        row.bhat(c, b);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s0 = add2(s0, v[e]);
          s1 = fma2(v[e], b[e], s1);
        }
      }
      n[0] = sum_of(s0), n[1] = sum_of(s1);
      block_sums(n, red);
      n[0] = A.layer ? n[0] * A.inv_cols : 0.0f;
      n[1] *= A.inv_cols;
    }
    for (int c = threadIdx.x * 8; c < A.cols; c += kWideThreads * 8) {
      f2 v[4], b[4];
      row.t(c, m[0], m[1], v);
      store_group8<T, false>(static_cast<T*>(A.dx) + r * A.lddx + c, A.cols - c, v);
      if (!A.dblock) continue;
      row.through(c, v);
      row.gated(c, v);
      if (A.block_gamma) {
        row.bhat(c, b);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = mul2(fma2(b[e], splat(-n[1]), add2(v[e], splat(-n[0]))), splat(row.block_rstd));
      }
      store_group8<T, false>(static_cast<T*>(A.dblock) + r * A.lddblock + c, A.cols - c, v);
    }
  }
}

// The parameters' gradients of one run of rows follow from four sums over them: of dy shat and dy, and of d bhat and d.
template <typename T>
__global__ void __launch_bounds__(kWideThreads) k_rn_param_wide(const BackwardArgs A, int64_t run) {
  in_turn();
  const int c = (blockIdx.x * kWideThreads + threadIdx.x) * 8;
  if (c >= A.cols) return;
  const Generator gen(A.drop);
  const int64_t r0 = blockIdx.y * run, r1 = r0 + run < A.rows ? r0 + run : A.rows;
  f2 sum[4][4] = {};
  for (int64_t r = r0; r < r1; ++r) {
    const RowBackward<T> row(A, gen, r);
    f2 v[4], b[4];
    if (A.gamma) {
      row.before(c, v, b);
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[0][e] = fma2(v[e], b[e], sum[0][e]), sum[1][e] = add2(sum[1][e], v[e]);
    }
    if (A.block_gamma || A.gate) {
      row.t(c, A.gamma ? A.sums[2 * r] : 0.0f, A.gamma ? A.sums[2 * r + 1] : 0.0f, v);
      row.through(c, v);
      row.bhat(c, b);
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[2][e] = fma2(v[e], b[e], sum[2][e]), sum[3][e] = add2(sum[3][e], v[e]);
    }
  }
  float* p = A.part + (int64_t)blockIdx.y * 4 * A.cols + c;
#pragma unroll
  for (int k = 0; k < 4; ++k, p += A.cols) store_group8<float, false>(p, A.cols - c, sum[k]);
}

// The parameters' gradients from the four sums of each part, added in order.
struct ParamGrads {
  void *dgamma, *dbeta, *dblock_gamma, *dblock_beta, *dgate;
};
template <typename G>
__global__ void __launch_bounds__(1024) k_rn_params(const float* __restrict__ part, int64_t parts, int cols, const float* __restrict__ block_gamma,
                                                    const float* __restrict__ block_beta, const float* __restrict__ gate, const ParamGrads out) {
  in_turn();
  __shared__ float red[32][33];
  const int lane = threadIdx.x & 31, row = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float total[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float s = 0.0f;
    if (c < cols) {
#pragma unroll 4
      for (int64_t p = row; p < parts; p += 32) s += part[(p * 4 + k) * cols + c];
    }
    red[row][lane] = s;
    __syncthreads();
    total[k] = warp_sum(red[lane][row]);  // of column `row` of the block
    __syncthreads();
  }
  const int o = blockIdx.x * 32 + row;
  if (lane != 0 || o >= cols) return;
  const float at = gate ? gate[o] : 1.0f;
  if (out.dgamma) static_cast<G*>(out.dgamma)[o] = from_f<G>(total[0]);
  if (out.dbeta) static_cast<G*>(out.dbeta)[o] = from_f<G>(total[1]);
  if (out.dblock_gamma) static_cast<G*>(out.dblock_gamma)[o] = from_f<G>(total[2] * at);
  if (out.dblock_beta) static_cast<G*>(out.dblock_beta)[o] = from_f<G>(total[3] * at);
  if (out.dgate) {
    const float g = block_gamma ? fmaf(total[2], block_gamma[o], block_beta ? total[3] * block_beta[o] : 0.0f) : total[2];
    static_cast<G*>(out.dgate)[o] = from_f<G>(g);
  }
}

unsigned at_most(int64_t want, int64_t per_sm) {
  const int64_t most = (int64_t)sm_count() * per_sm;
  return (unsigned)(want < most ? want : most);
}

template <typename T>
cudaError_t forward(const ForwardArgs& a, cudaStream_t s) {
  return launch_after(k_rn_forward_wide<T>, at_most(a.rows, 8), kWideThreads, s, a);
}

// The runs of rows that each leave a part of the parameters' sums.
int64_t rows_a_part(int64_t rows) { return ceil_div(rows, 64); }

// Takes the workspace; with `run`, enqueues the work too.
template <typename T>
cudaError_t backward(BackwardArgs a, const ParamGrads& g, int32_t grad_dtype, char* workspace, int64_t* used, cudaStream_t s, bool run) {
  const bool params = g.dgamma || g.dbeta || g.dblock_gamma || g.dblock_beta || g.dgate;
  const int64_t run_rows = a.rows ? rows_a_part(a.rows) : 1, parts = params ? ceil_div(a.rows, run_rows) : 0;
  const int64_t part_bytes = (parts * 4 * a.cols * 4 + 15) & ~(int64_t)15;
  *used = part_bytes + (a.gamma ? a.rows * 8 : 0);
  if (!run) return cudaSuccess;
  a.part = reinterpret_cast<float*>(workspace);
  a.sums = reinterpret_cast<float*>(workspace + part_bytes);
  cudaError_t e = cudaSuccess;
  if (a.rows > 0) e = launch_after(k_rn_backward_wide<T>, at_most(a.rows, 8), kWideThreads, s, a);
  if (e == cudaSuccess && parts > 0)
    e = launch_after(k_rn_param_wide<T>, dim3((unsigned)ceil_div(a.cols, kWideThreads * 8), (unsigned)parts), kWideThreads, s, a, run_rows);
  if (e != cudaSuccess || !params) return e;
  auto finish = [&](auto* kernel) {
    return launch_after(kernel, (unsigned)ceil_div(a.cols, 32), 1024, s, a.part, parts, a.cols, a.block_gamma, a.block_beta, a.gate, g);
  };
  return grad_dtype == ONEBIT_F32 ? finish(k_rn_params<float>) : grad_dtype == ONEBIT_F16 ? finish(k_rn_params<__half>) : finish(k_rn_params<__nv_bfloat16>);
}

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
  const BackwardArgs b{a.dy, a.lddy, a.ds, a.ldds, a.s, a.lds, a.block, a.ldblock, a.gamma, a.block_gamma, a.block_beta, a.gate, drop, a.mean, a.rstd,
                       a.block_mean, a.block_rstd, a.dx, a.lddx, a.dblock, a.lddblock, a.rows, (int)a.cols, (int)ceil_div(a.cols, 8),
                       a.norm == ONEBIT_NORM_LAYER, 1.0f / (float)a.cols, a.scale, nullptr, nullptr};
  const ParamGrads g{a.dgamma, a.dbeta, a.dblock_gamma, a.dblock_beta, a.dgate};
  return a.dtype == ONEBIT_F32   ? backward<float>(b, g, a.grad_dtype, workspace, used, s, run)
         : a.dtype == ONEBIT_F16 ? backward<__half>(b, g, a.grad_dtype, workspace, used, s, run)
                                 : backward<__nv_bfloat16>(b, g, a.grad_dtype, workspace, used, s, run);
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
  const ForwardArgs f{a.x, a.ldx, a.block, a.ldblock, a.gamma, a.beta, a.block_gamma, a.block_beta, a.gate, drop, a.s, a.lds, a.y, a.ldy, a.mean, a.rstd,
                      a.block_mean, a.block_rstd, a.rows, (int)a.cols, (int)ceil_div(a.cols, 8), a.norm == ONEBIT_NORM_LAYER, 1.0f / (float)a.cols,
                      a.eps, a.scale};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = a.dtype == ONEBIT_F32 ? forward<float>(f, s) : a.dtype == ONEBIT_F16 ? forward<__half>(f, s) : forward<__nv_bfloat16>(f, s);
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
