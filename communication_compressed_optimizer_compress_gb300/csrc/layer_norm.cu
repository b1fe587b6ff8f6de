// layer_norm.cu -- layer norm over the columns of each row, forward and backward, with the gradients
// of gamma and beta.  See include/onebit_layers.h for the formulas.
#include <type_traits>

#include "layers_common.cuh"

namespace onebit {
namespace layers {
namespace {

// Both passes are bound by the bytes of the rows.  A row is held in registers between its statistics and
// its output, so that it is read once: TPR threads have a row, a thread CH groups of eight columns (and
// the same columns of every row that it meets, so that the parameters' gradients add up in registers too).  Widths are
// served by the narrowest of the forms below; a wider row than the widest takes the re-reading kernels.
//
// In the wide form (VEC: rows on 16 bytes, a multiple of eight columns) a group is eight columns that lie
// together; otherwise it is columns lane and lane + 32 of four runs of 64, so that single-element accesses
// of a warp are contiguous and a run is still one block of the 8-bit checkpoint.
template <int TPR, bool VEC>
struct Columns {
  static constexpr int kWarps = TPR / 32;
  __device__ static __forceinline__ int at(int t, int j, int e) {
    return VEC ? (j * TPR + t) * 8 + e : ((j * 4 + e / 2) * kWarps + t / 32) * 64 + (t & 31) + 32 * (e & 1);
  }
};

template <typename T, int TPR, int CH, bool VEC>
struct RowInput;  // a row's columns of one thread, as they lie in memory
template <typename T, int TPR, int CH>
struct RowInput<T, TPR, CH, true> {
  Raw8<T> raw[CH];
  __device__ __forceinline__ void load(const T* p, int t, int cols) {
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int c = Columns<TPR, true>::at(t, j, 0);
      if (c < cols) raw[j] = load8(p + c);
      else raw[j] = Raw8<T>{};
    }
  }
  __device__ __forceinline__ void expand(int j, float* f) const { expand8(raw[j], f); }
};
template <typename T, int TPR, int CH>
struct RowInput<T, TPR, CH, false> {
  T raw[CH][8];
  __device__ __forceinline__ void load(const T* p, int t, int cols) {
#pragma unroll
    for (int j = 0; j < CH; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = Columns<TPR, false>::at(t, j, e);
        raw[j][e] = c < cols ? p[c] : from_f<T>(0.0f);
      }
  }
  __device__ __forceinline__ void expand(int j, float* f) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = to_f(raw[j][e]);
  }
};
template <typename T, int TPR, bool VEC>
__device__ __forceinline__ void store_group(T* p, int t, int j, int cols, const float* f) {
  if (VEC) {
    const int c = Columns<TPR, true>::at(t, j, 0);
    if (c < cols) store8(p + c, f);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = Columns<TPR, false>::at(t, j, e);
      if (c < cols) p[c] = from_f<T>(f[e]);
    }
  }
}

// gamma or beta of a group, 0 past the end: from L1, where it stays for every row
template <int TPR, bool VEC>
__device__ __forceinline__ void param_group(const float* p, int t, int j, int cols, float* f) {
  if (VEC) {
    const int c = Columns<TPR, true>::at(t, j, 0);
    const Raw8<float> r = c < cols ? load8(p + c) : Raw8<float>{};
    expand8(r, f);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = Columns<TPR, false>::at(t, j, e);
      f[e] = c < cols ? __ldg(p + c) : 0.0f;
    }
  }
}

// Sums over the TPR threads of a row, the same order on every call; every thread gets them.  `red` has
// room for two sets, used alternately, so that one barrier a call is enough.
template <int TPR, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*red)[N * 32], int& turn, int bar) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
  if (TPR == 32) return;
  float* r = red[turn];
  turn ^= 1;
  const int warp = (threadIdx.x % TPR) >> 5;
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) r[warp * N + i] = v[i];
  }
  asm volatile("bar.sync %0, %1;" ::"r"(bar), "n"(TPR) : "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = 0.0f;
#pragma unroll
    for (int w = 0; w < TPR / 32; ++w) v[i] += r[w * N + i];
  }
}

struct ForwardArgs {
  const void* x;
  int64_t ldx, rows;
  int cols, blocks;
  float inv_cols, eps;
  const float *gamma, *beta;
  void* y;
  int64_t ldy;
  float *mean, *rstd;
  int8_t* codes;
  float* scales;
};

template <int TPR>
constexpr int kForwardThreads = TPR < 128 ? 128 : TPR;

template <typename T, int TPR, int CH, bool VEC>
__global__ void __launch_bounds__(kForwardThreads<TPR>, (CH > 1 ? TPR < 512 ? 768 : 512 : 1536) / kForwardThreads<TPR>) k_ln_forward(const ForwardArgs A) {
  constexpr int kGroups = kForwardThreads<TPR> / TPR;
  using Col = Columns<TPR, VEC>;
  __shared__ float red[2][32];
  const int t = threadIdx.x % TPR;
  const int64_t first = (int64_t)blockIdx.x * kGroups + threadIdx.x / TPR, step = (int64_t)gridDim.x * kGroups;
  int turn = 0;
  RowInput<T, TPR, CH, VEC> in;
  if (first < A.rows) in.load(static_cast<const T*>(A.x) + first * A.ldx, t, A.cols);
  for (int64_t r = first; r < A.rows; r += step) {
    float x[CH][8];
#pragma unroll
    for (int j = 0; j < CH; ++j) in.expand(j, x[j]);
    if (r + step < A.rows) in.load(static_cast<const T*>(A.x) + (r + step) * A.ldx, t, A.cols);  // under this row's work
    float s[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < CH; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) s[0] += x[j][e];
    row_sums<TPR>(s, red, turn, 1);
    const float mean = s[0] * A.inv_cols;
    s[0] = 0.0f;
#pragma unroll
    for (int j = 0; j < CH; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = Col::at(t, j, e) < A.cols ? x[j][e] - mean : 0.0f;
        s[0] = fmaf(d, d, s[0]);
      }
    row_sums<TPR>(s, red, turn, 1);
    const float rstd = 1.0f / sqrtf(fmaf(s[0], A.inv_cols, A.eps));
    if (t == 0) {
      A.mean[r] = mean;
      A.rstd[r] = rstd;
    }
    if (A.codes) {
      int8_t* codes = A.codes + r * A.cols;
      float* scales = A.scales + r * A.blocks;
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        if (VEC) {  // a block is eight neighbouring lanes
          const int c = Col::at(t, j, 0);
          float most = 0.0f;
#pragma unroll
          for (int e = 0; e < 8; ++e) most = max_nan(most, fabsf(x[j][e]));
#pragma unroll
          for (int o = 1; o < 8; o *= 2) most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, o));
          const BlockScale q = block_scale(most);
          if (c < A.cols) {
            *reinterpret_cast<uint2*>(codes + c) = make_uint2(codes4(x[j][0], x[j][1], x[j][2], x[j][3], q.inv), codes4(x[j][4], x[j][5], x[j][6], x[j][7], q.inv));
            if ((t & 7) == 0) scales[c / kBlock] = q.scale;
          }
        } else {  // a block is two columns of every lane
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const int c = Col::at(t, j, e), c0 = c - (t & 31);
            if (c0 >= A.cols) continue;
            const BlockScale q = block_scale(warp_max_nan(max_nan(fabsf(x[j][e]), fabsf(x[j][e + 1]))));
            if (c < A.cols) codes[c] = (int8_t)code_of(x[j][e], q.inv);
            if (c + 32 < A.cols) codes[c + 32] = (int8_t)code_of(x[j][e + 1], q.inv);
            if ((t & 31) == 0) scales[c0 / kBlock] = q.scale;
          }
        }
      }
    }
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      float y[8], g[8], b[8];
      param_group<TPR, VEC>(A.gamma, t, j, A.cols, g);
      param_group<TPR, VEC>(A.beta, t, j, A.cols, b);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = fmaf((x[j][e] - mean) * rstd, g[e], b[e]);
      store_group<T, TPR, VEC>(static_cast<T*>(A.y) + r * A.ldy, t, j, A.cols, y);
    }
  }
}

struct BackwardArgs {
  const void* dy;
  int64_t lddy;
  const void* x;  // the layer's input, or its 8-bit checkpoint
  int64_t ldx;
  const int8_t* codes;
  const float* scales;
  int64_t rows;
  int cols, blocks;
  float inv_cols;
  const float *gamma, *mean, *rstd;
  const void* add;
  int64_t ldadd;
  void* dx;
  int64_t lddx;
  void *dgamma, *dbeta;
  int32_t grad_dtype;
  float* part;  // [block][2][cols]
};

template <int TPR>
constexpr int kBackThreads = TPR < 256 ? 256 : TPR;

// The kept input of one thread's columns: values, or codes with the scale of their block.
template <typename T, int TPR, int CH, bool VEC, bool CODES>
struct KeptRow;
template <typename T, int TPR, int CH, bool VEC>
struct KeptRow<T, TPR, CH, VEC, false> {
  RowInput<T, TPR, CH, VEC> in;
  __device__ __forceinline__ void load(const BackwardArgs& A, int64_t r, int t) { in.load(static_cast<const T*>(A.x) + r * A.ldx, t, A.cols); }
  __device__ __forceinline__ void expand(int j, float* f) const { in.expand(j, f); }
};
template <typename T, int TPR, int CH>
struct KeptRow<T, TPR, CH, true, true> {
  uint2 raw[CH];
  float scale[CH];
  __device__ __forceinline__ void load(const BackwardArgs& A, int64_t r, int t) {
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int c = Columns<TPR, true>::at(t, j, 0);
      raw[j] = c < A.cols ? __ldg(reinterpret_cast<const uint2*>(A.codes + r * A.cols + c)) : make_uint2(0, 0);
      scale[j] = c < A.cols ? __ldg(A.scales + r * A.blocks + c / kBlock) : 0.0f;
    }
  }
  __device__ __forceinline__ void expand(int j, float* f) const {
    values4<T>(raw[j].x, scale[j], f);
    values4<T>(raw[j].y, scale[j], f + 4);
  }
};
template <typename T, int TPR, int CH>
struct KeptRow<T, TPR, CH, false, true> {
  int8_t raw[CH][8];
  float scale[CH][4];
  __device__ __forceinline__ void load(const BackwardArgs& A, int64_t r, int t) {
#pragma unroll
    for (int j = 0; j < CH; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = Columns<TPR, false>::at(t, j, e);
        raw[j][e] = c < A.cols ? A.codes[r * A.cols + c] : (int8_t)0;
        if ((e & 1) == 0) scale[j][e / 2] = c < A.cols ? A.scales[r * A.blocks + c / kBlock] : 0.0f;
      }
  }
  __device__ __forceinline__ void expand(int j, float* f) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = value_of<T>(raw[j][e], scale[j][e / 2]);
  }
};

// dx of every row, and this block's share of dgamma and dbeta.  Each thread adds up its own columns over
// the rows that it meets; at the end the block's row groups are joined in shared memory, in order.
template <typename T, int TPR, int CH, bool VEC, bool CODES>
__global__ void __launch_bounds__(kBackThreads<TPR>, TPR < 256 ? 3 : 1) k_ln_backward(const BackwardArgs A) {
  constexpr int kGroups = kBackThreads<TPR> / TPR;
  using Col = Columns<TPR, VEC>;
  __shared__ float red[kGroups][2][2 * 32];
  __shared__ float join[kGroups == 1 ? 1 : 2 * TPR * CH * 8];
  const int t = threadIdx.x % TPR, group = threadIdx.x / TPR;
  const int64_t first = (int64_t)blockIdx.x * kGroups + group, step = (int64_t)gridDim.x * kGroups;
  int turn = 0;
  launch_next();
  float dg[CH][8], db[CH][8];
#pragma unroll
  for (int j = 0; j < CH; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) dg[j][e] = db[j][e] = 0.0f;
  KeptRow<T, TPR, CH, VEC, CODES> kept;
  RowInput<T, TPR, CH, VEC> dyin, addin, addnow;
  float mu = 0.0f, rs = 0.0f;
  auto load = [&](int64_t r) {
    kept.load(A, r, t);
    dyin.load(static_cast<const T*>(A.dy) + r * A.lddy, t, A.cols);
    if (A.add) addin.load(static_cast<const T*>(A.add) + r * A.ldadd, t, A.cols);
    mu = __ldg(A.mean + r);
    rs = __ldg(A.rstd + r);
  };
  if (first < A.rows) load(first);
  for (int64_t r = first; r < A.rows; r += step) {
    float xh[CH][8], d[CH][8];
    const float rstd = rs;
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      float gamma[8];
      param_group<TPR, VEC>(A.gamma, t, j, A.cols, gamma);
      kept.expand(j, xh[j]);
      dyin.expand(j, d[j]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        // columns past the end have dy = gamma = 0 and add nothing
        xh[j][e] = (xh[j][e] - mu) * rstd;
        dg[j][e] = fmaf(d[j][e], xh[j][e], dg[j][e]);
        db[j][e] += d[j][e];
        d[j][e] *= gamma[e];
        s[0] += d[j][e];
        s[1] = fmaf(d[j][e], xh[j][e], s[1]);
      }
    }
    if (A.add) addnow = addin;
    if (r + step < A.rows) load(r + step);  // under this row's sums
    row_sums<TPR>(s, red[group], turn, 1 + group);
    s[0] *= A.inv_cols;
    s[1] *= A.inv_cols;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      float o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = rstd * (d[j][e] - s[0] - xh[j][e] * s[1]);
      if (A.add) {
        float a[8];
        addnow.expand(j, a);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] += a[e];
      }
      store_group<T, TPR, VEC>(static_cast<T*>(A.dx) + r * A.lddx, t, j, A.cols, o);
    }
  }
  if (kGroups > 1) {
    for (int q = 0; q < kGroups; ++q) {
      __syncthreads();
      if (group == q) {
#pragma unroll
        for (int j = 0; j < CH; ++j)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int i = (j * 8 + e) * TPR + t;
            join[i] = q ? join[i] + dg[j][e] : dg[j][e];
            join[TPR * CH * 8 + i] = q ? join[TPR * CH * 8 + i] + db[j][e] : db[j][e];
          }
      }
    }
    __syncthreads();
  }
  if (group == 0) {
    float* p = A.part + (int64_t)blockIdx.x * 2 * A.cols;
#pragma unroll
    for (int j = 0; j < CH; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = Col::at(t, j, e), i = (j * 8 + e) * TPR + t;
        if (c < A.cols) {
          p[c] = kGroups > 1 ? join[i] : dg[j][e];
          p[A.cols + c] = kGroups > 1 ? join[TPR * CH * 8 + i] : db[j][e];
        }
      }
  }
}

// Rows too wide for registers: read again for each step, one block a row.
constexpr int kLnThreads = 256;
constexpr int kLnWarps = kLnThreads / 32;
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

template <typename T>
__global__ void __launch_bounds__(kLnThreads) k_ln_forward_wide(const ForwardArgs A) {
  __shared__ float red[kLnWarps];
  for (int64_t r = blockIdx.x; r < A.rows; r += gridDim.x) {
    const T* xr = static_cast<const T*>(A.x) + r * A.ldx;
    T* yr = static_cast<T*>(A.y) + r * A.ldy;
    float s = 0.0f;
    for (int c = threadIdx.x; c < A.cols; c += kLnThreads) s += to_f(xr[c]);
    const float mean = block_sum(s, red) * A.inv_cols;
    s = 0.0f;
    for (int c = threadIdx.x; c < A.cols; c += kLnThreads) {
      const float d = to_f(xr[c]) - mean;
      s = fmaf(d, d, s);
    }
    const float rstd = 1.0f / sqrtf(fmaf(block_sum(s, red), A.inv_cols, A.eps));
    for (int c = threadIdx.x; c < A.cols; c += kLnThreads)
      yr[c] = from_f<T>(fmaf((to_f(xr[c]) - mean) * rstd, A.gamma[c], A.beta[c]));
    if (threadIdx.x == 0) {
      A.mean[r] = mean;
      A.rstd[r] = rstd;
    }
    if (A.codes) {
      const int lane = threadIdx.x & 31;
      for (int b = threadIdx.x >> 5; b < A.blocks; b += kLnWarps) {
        const int c0 = b * kBlock + lane, c1 = c0 + 32;
        const float v0 = c0 < A.cols ? to_f(xr[c0]) : 0.0f, v1 = c1 < A.cols ? to_f(xr[c1]) : 0.0f;
        const BlockScale q = block_scale(warp_max_nan(max_nan(fabsf(v0), fabsf(v1))));
        if (c0 < A.cols) A.codes[r * A.cols + c0] = (int8_t)code_of(v0, q.inv);
        if (c1 < A.cols) A.codes[r * A.cols + c1] = (int8_t)code_of(v1, q.inv);
        if (lane == 0) A.scales[r * A.blocks + b] = q.scale;
      }
    }
  }
}

template <typename T>
__device__ __forceinline__ float kept_at(const BackwardArgs& A, int64_t r, int c) {
  return A.codes ? value_of<T>(A.codes[r * A.cols + c], A.scales[r * A.blocks + c / kBlock]) : to_f(static_cast<const T*>(A.x)[r * A.ldx + c]);
}
template <typename T>
__global__ void __launch_bounds__(kLnThreads) k_ln_backward_wide(const BackwardArgs A) {
  __shared__ float red[kLnWarps];
  const T *dy = static_cast<const T*>(A.dy), *add = static_cast<const T*>(A.add);
  for (int64_t r = blockIdx.x; r < A.rows; r += gridDim.x) {
    const float mu = A.mean[r], rs = A.rstd[r];
    float s1 = 0.0f, s2 = 0.0f;
    for (int c = threadIdx.x; c < A.cols; c += kLnThreads) {
      const float g = to_f(dy[r * A.lddy + c]) * A.gamma[c];
      s1 += g;
      s2 = fmaf(g, (kept_at<T>(A, r, c) - mu) * rs, s2);
    }
    s1 = block_sum(s1, red) * A.inv_cols;
    s2 = block_sum(s2, red) * A.inv_cols;
    for (int c = threadIdx.x; c < A.cols; c += kLnThreads) {
      const float g = to_f(dy[r * A.lddy + c]) * A.gamma[c];
      float d = rs * (g - s1 - (kept_at<T>(A, r, c) - mu) * rs * s2);
      if (add) d += to_f(add[r * A.ldadd + c]);
      static_cast<T*>(A.dx)[r * A.lddx + c] = from_f<T>(d);
    }
  }
}
// this block's rows' share of dgamma and dbeta
template <typename T>
__global__ void __launch_bounds__(kLnThreads) k_ln_param_wide(const BackwardArgs A, int64_t run) {
  const int c = blockIdx.x * kLnThreads + threadIdx.x;
  if (c >= A.cols) return;
  const int64_t r0 = blockIdx.y * run, r1 = r0 + run < A.rows ? r0 + run : A.rows;
  float g = 0.0f, b = 0.0f;
  for (int64_t r = r0; r < r1; ++r) {
    const float d = to_f(static_cast<const T*>(A.dy)[r * A.lddy + c]);
    g = fmaf(d, (kept_at<T>(A, r, c) - A.mean[r]) * A.rstd[r], g);
    b += d;
  }
  float* p = A.part + (int64_t)blockIdx.y * 2 * A.cols;
  p[c] = g;
  p[A.cols + c] = b;
}

unsigned at_most(int64_t want, int64_t per_sm) {
  const int64_t most = (int64_t)sm_count() * per_sm;
  return (unsigned)(want < most ? want : most);
}

// the widest row of the forward and backward forms that hold rows in registers
constexpr int kForwardCols = 512 * 4 * 8, kBackwardCols = 512 * 2 * 8;

template <typename T, bool VEC>
void launch_forward(const ForwardArgs& a, cudaStream_t s) {
  auto go = [&](auto tpr, auto ch, int per_sm) {
    constexpr int kTpr = decltype(tpr)::value, kCh = decltype(ch)::value, kThreads = kForwardThreads<kTpr>;
    k_ln_forward<T, kTpr, kCh, VEC><<<at_most(ceil_div(a.rows, kThreads / kTpr), per_sm), kThreads, 0, s>>>(a);
  };
  using std::integral_constant;
  if (a.cols <= 256) go(integral_constant<int, 32>{}, integral_constant<int, 1>{}, 12);
  else if (a.cols <= 1024) go(integral_constant<int, 32>{}, integral_constant<int, 4>{}, 6);
  else if (a.cols <= 4096) go(integral_constant<int, 128>{}, integral_constant<int, 4>{}, 6);
  else if (a.cols <= kForwardCols) go(integral_constant<int, 512>{}, integral_constant<int, 4>{}, 1);
  else k_ln_forward_wide<T><<<at_most(a.rows, 8), kLnThreads, 0, s>>>(a);
}

// Blocks of the backward kernel, which are the parts that the parameters' gradients are summed from.
int backward_parts(int64_t rows, int64_t cols) {
  if (rows == 0) return 0;
  if (cols > kBackwardCols) return (int)ceil_div(rows, ceil_div(rows, 64));
  const int tpr = cols <= 256 ? 32 : cols <= 1024 ? 128 : 512;
  return (int)at_most(ceil_div(rows, tpr < 256 ? 256 / tpr : 1), tpr < 256 ? 3 : 1);
}

template <typename T, bool VEC, bool CODES>
void launch_backward(const BackwardArgs& a, int parts, cudaStream_t s) {
  if (a.cols <= 256) k_ln_backward<T, 32, 1, VEC, CODES><<<parts, kBackThreads<32>, 0, s>>>(a);
  else if (a.cols <= 1024) k_ln_backward<T, 128, 1, VEC, CODES><<<parts, kBackThreads<128>, 0, s>>>(a);
  else if (a.cols <= 4096) k_ln_backward<T, 512, 1, VEC, CODES><<<parts, kBackThreads<512>, 0, s>>>(a);
  else k_ln_backward<T, 512, 2, VEC, CODES><<<parts, kBackThreads<512>, 0, s>>>(a);
}

template <typename T>
cudaError_t launch_backward(const BackwardArgs& a, cudaStream_t s) {
  const int parts = backward_parts(a.rows, a.cols);
  auto on16 = [](const void* p, int64_t ld) { return aligned(p, 16) && (ld * (int64_t)sizeof(T)) % 16 == 0; };
  const bool vec = a.cols % 8 == 0 && on16(a.dy, a.lddy) && on16(a.x, a.ldx) && on16(a.add, a.ldadd) && on16(a.dx, a.lddx) && aligned(a.codes, 8);
  if (parts == 0) {  // no rows
  } else if (a.cols > kBackwardCols) {
    k_ln_backward_wide<T><<<at_most(a.rows, 8), kLnThreads, 0, s>>>(a);
    k_ln_param_wide<T><<<dim3((unsigned)ceil_div(a.cols, kLnThreads), (unsigned)parts), kLnThreads, 0, s>>>(a, ceil_div(a.rows, 64));
  } else if (vec) {
    if (a.codes) launch_backward<T, true, true>(a, parts, s);
    else launch_backward<T, true, false>(a, parts, s);
  } else {
    if (a.codes) launch_backward<T, false, true>(a, parts, s);
    else launch_backward<T, false, false>(a, parts, s);
  }
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? sum_parts(a.grad_dtype, a.part, parts, 2 * (int64_t)a.cols, a.cols, a.dgamma, a.dbeta, s) : e;
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
  const ForwardArgs a{x, ldx, rows, (int)cols, (int)blocks, 1.0f / (float)cols, eps, gamma, beta, y, ldy, mean, rstd, codes, scales};
  const bool vec = cols % 8 == 0 && aligned(x, 16) && aligned(y, 16) && (ldx * e) % 16 == 0 && (ldy * e) % 16 == 0 && aligned(codes, 8);
  auto go = [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    if (vec) launch_forward<T, true>(a, s);
    else launch_forward<T, false>(a, s);
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
  *bytes = (size_t)((int64_t)backward_parts(rows, cols) * 2 * cols * 4);
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
  const BackwardArgs a{dy, lddy, x, ldx, codes, scales, rows, (int)cols, (int)blocks, 1.0f / (float)cols, gamma, mean, rstd, add, ldadd, dx, lddx,
                       dgamma, dbeta, grad_dtype, static_cast<float*>(workspace)};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t ce = dtype == ONEBIT_F32 ? launch_backward<float>(a, s)
                         : dtype == ONEBIT_F16 ? launch_backward<__half>(a, s)
                                               : launch_backward<__nv_bfloat16>(a, s);
  return ce == cudaSuccess ? ONEBIT_OK : cuda_fail(ce, "onebit_layer_norm_backward");
}
