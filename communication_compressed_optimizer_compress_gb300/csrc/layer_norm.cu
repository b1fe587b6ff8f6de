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
// In the wide form (VEC: rows, gamma and beta on 16 bytes, a multiple of eight columns) a group is eight columns that
// lie together; otherwise it is columns lane and lane + 32 of four runs of 64, so that single-element accesses
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
  __device__ __forceinline__ void expand(int j, f2* f) const { expand8(raw[j], f); }
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
  __device__ __forceinline__ void expand(int j, f2* f) const {
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = pair(to_f(raw[j][2 * e]), to_f(raw[j][2 * e + 1]));
  }
};
template <typename T, int TPR, bool VEC>
__device__ __forceinline__ void store_group(T* p, int t, int j, int cols, const f2* f) {
  if (VEC) {
    const int c = Columns<TPR, true>::at(t, j, 0);
    if (c < cols) store8(p + c, f);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {  // columns c and c + 32
      const int c = Columns<TPR, false>::at(t, j, 2 * e);
      const float2 h = halves(f[e]);
      if (c < cols) p[c] = from_f<T>(h.x);
      if (c + 32 < cols) p[c + 32] = from_f<T>(h.y);
    }
  }
}

// gamma or beta of a group, 0 past the end: from L1, where it stays for every row
template <int TPR, bool VEC>
__device__ __forceinline__ void param_group(const float* p, int t, int j, int cols, f2* f) {
  if (VEC) {
    const int c = Columns<TPR, true>::at(t, j, 0);
    const Raw8<float> r = c < cols ? load8(p + c) : Raw8<float>{};
    expand8(r, f);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = Columns<TPR, false>::at(t, j, 2 * e);
      f[e] = pair(c < cols ? __ldg(p + c) : 0.0f, c + 32 < cols ? __ldg(p + c + 32) : 0.0f);
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
constexpr int kForwardThreads = TPR < 128 ? 128 / TPR * TPR : TPR;
template <typename T, int TPR, int CH, bool VEC>
constexpr int kForwardRoom = VEC && sizeof(T) == 2 && CH == 1 && TPR > 64 ? 1024 : TPR < 256 && !(TPR == 32 && CH == 2) ? 640 : 512;  // threads an SM

// NR rows at a time (1 or 2): their sums go through the shuffles and the barrier together.  gamma and beta stay in registers
// where they fit beside the rows; elsewhere they are read (from L1) once for the NR rows.  16384 x 1024 bf16 with the
// checkpoint: a warp a row, which reads them for every row, 18.6 us (62% of the L1's cycles), 128 threads a row that hold
// them 17.2, at 1024 threads an SM (18.5 at 640); 33 rows 2.7 and 2.1 us.
template <typename T, int TPR, int CH, int NR, bool VEC, bool FULL>
__global__ void __launch_bounds__(kForwardThreads<TPR>, kForwardRoom<T, TPR, CH, VEC> / kForwardThreads<TPR>) k_ln_forward(const ForwardArgs A) {
  static_assert(NR == 1 || NR == 2, "rows at a time");
  in_turn();
  constexpr int kGroups = kForwardThreads<TPR> / TPR;
  const int cols = FULL ? TPR * CH * 8 : A.cols;
  using Col = Columns<TPR, VEC>;
  __shared__ float red[kGroups][2][NR * 32];
  const int t = threadIdx.x % TPR, group = threadIdx.x / TPR;
  const int64_t first = ((int64_t)blockIdx.x * kGroups + group) * NR, step = (int64_t)gridDim.x * kGroups * NR;
  int turn = 0;
  RowInput<T, TPR, CH, VEC> in[NR];
  const T* px = static_cast<const T*>(A.x) + first * A.ldx;
  T* py = static_cast<T*>(A.y) + first * A.ldy;
  auto load = [&](int64_t r) {
#pragma unroll
    for (int n = 0; n < NR; ++n)
      if (r + n < A.rows) in[n].load(px + n * A.ldx, t, cols);
  };
  load(first);
  // (in the single-element forms they would spill: 16384 x 1155 bf16 with the checkpoint 60 us for 48.5; in the wide form
  // of 2048 columns 17.7 for 17.1)
  constexpr bool kHold = VEC && (CH == 1 || (CH == 2 && TPR == 256 && sizeof(T) == 2));
  f2 gs[kHold ? CH : 1][4], bs[kHold ? CH : 1][4];
  if (kHold) {
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      param_group<TPR, VEC>(A.gamma, t, j, cols, gs[kHold ? j : 0]);
      param_group<TPR, VEC>(A.beta, t, j, cols, bs[kHold ? j : 0]);
    }
  }
  for (int64_t r = first; r < A.rows; r += step) {
    f2 x[NR][CH][4];
    float mean[NR], rstd[NR];
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int j = 0; j < CH; ++j) in[n].expand(j, x[n][j]);
    px += step * A.ldx;
    load(r + step);  // under these rows' work
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      f2 s = 0;
#pragma unroll
      for (int j = 0; j < CH; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) s = add2(s, x[n][j][e]);
      mean[n] = sum_of(s);
    }
    row_sums<TPR>(mean, red[group], turn, 1 + group);
    if (A.codes) {
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        if (r + n >= A.rows) continue;
        int8_t* codes = A.codes + (r + n) * cols;
        float* scales = A.scales + (r + n) * A.blocks;
#pragma unroll
        for (int j = 0; j < CH; ++j) {
          const f2* v = x[n][j];
          if (VEC) {  // a block is eight neighbouring lanes
            const int c = Col::at(t, j, 0);
            float most = 0.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e) most = max_abs(most, v[e]);
#pragma unroll
            for (int o = 1; o < 8; o *= 2) most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, o));
            const BlockScale q = block_scale(most);
            if (c < cols) {
              *reinterpret_cast<uint2*>(codes + c) = make_uint2(codes4(v[0], v[1], q.inv), codes4(v[2], v[3], q.inv));
              if ((t & 7) == 0) scales[c / kBlock] = q.scale;
            }
          } else {  // a block is two columns of every lane
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int c = Col::at(t, j, 2 * e), c0 = c - (t & 31);
              if (c0 >= cols) continue;
              const BlockScale q = block_scale(warp_max_nan(max_abs(0.0f, v[e])));
              const float2 h = halves(v[e]);
              if (c < cols) codes[c] = (int8_t)code_of(h.x, q.inv);
              if (c + 32 < cols) codes[c + 32] = (int8_t)code_of(h.y, q.inv);
              if ((t & 31) == 0) scales[c0 / kBlock] = q.scale;
            }
          }
        }
      }
    }
    // from here on x is its distance from the mean
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      mean[n] *= A.inv_cols;
      f2 s = 0;
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        const f2 shift = VEC && Col::at(t, j, 0) >= cols ? 0 : splat(-mean[n]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int c = Col::at(t, j, 2 * e);
          x[n][j][e] = add2(x[n][j][e], VEC ? shift : pair(c < cols ? -mean[n] : 0.0f, c + 32 < cols ? -mean[n] : 0.0f));
          s = fma2(x[n][j][e], x[n][j][e], s);
        }
      }
      rstd[n] = sum_of(s);
    }
    row_sums<TPR>(rstd, red[group], turn, 1 + group);
#pragma unroll
    for (int n = 0; n < NR; n += 2) {
      const float2 v = halves(rsqrt_rounded(fma2(pair(rstd[n], rstd[NR - 1]), splat(A.inv_cols), splat(A.eps))));
      rstd[n] = v.x, rstd[NR - 1] = NR > 1 ? v.y : v.x;
    }
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      if (t == 0 && r + n < A.rows) {
        A.mean[r + n] = mean[n];
        A.rstd[r + n] = rstd[n];
      }
    }
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      f2 g[4], b[4];
      if (kHold) {
#pragma unroll
        for (int e = 0; e < 4; ++e) g[e] = gs[kHold ? j : 0][e], b[e] = bs[kHold ? j : 0][e];
      } else {
        param_group<TPR, VEC>(A.gamma, t, j, cols, g);
        param_group<TPR, VEC>(A.beta, t, j, cols, b);
      }
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        f2 y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = fma2(mul2(x[n][j][e], splat(rstd[n])), g[e], b[e]);
        if (r + n < A.rows) store_group<T, TPR, VEC>(py + n * A.ldy, t, j, cols, y);
      }
    }
    py += step * A.ldy;
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

// Threads that an SM has registers for (96 a thread, 128 with two groups of columns), in as few blocks as can be: a
// block leaves one partial sum of each parameter.  (With 768 threads of 80 registers the single-element forms spill:
// 16384 x 1001 bf16 57.7 us for 44.0.)
template <int CH>
constexpr int kBackRoom = CH == 1 ? 640 : 512;
template <int TPR, int CH>
constexpr int kBackGroups = kBackRoom<CH> / TPR < 10 ? kBackRoom<CH> / TPR : 10;  // rows at a time
template <int TPR, int CH>
constexpr int kBackThreads = TPR * kBackGroups<TPR, CH>;

// The kept input of one thread's columns: values, or codes with the scale of their block.  normal() gives
// the normalised values (x - mean) rstd.  The difference comes first, where it is exact or nearly so: x rstd - mean rstd,
// one operation less, takes its error from the size of the mean (|mean| of 1000 standard deviations: 2e-5 of the
// normalised value, 3e-8 this way).
//
// From codes by one fused operation and a product.  In fp32 a code times its scale can round past the largest value
// (value_of()); there both factors of the product are moved by a power of two.
template <typename T>
__device__ __forceinline__ f2 normal_of_codes(f2 codes, float scale, float mean, float rstd) {
  constexpr float kDown = sizeof(T) == 4 ? 0.5f : 1.0f, kUp = sizeof(T) == 4 ? 2.0f : 1.0f;
  return mul2(fma2(codes, splat(scale * kDown), splat(-mean * kDown)), splat(rstd * kUp));
}
template <typename T, int TPR, int CH, bool VEC, bool CODES>
struct KeptRow;
template <typename T, int TPR, int CH, bool VEC>
struct KeptRow<T, TPR, CH, VEC, false> {
  RowInput<T, TPR, CH, VEC> in;
  const T* p;
  int64_t step;
  __device__ __forceinline__ KeptRow(const BackwardArgs& A, int64_t first, int64_t rows) : p(static_cast<const T*>(A.x) + first * A.ldx), step(rows * A.ldx) {}
  __device__ __forceinline__ void load(int t, int cols) {
    in.load(p, t, cols);
    p += step;
  }
  __device__ __forceinline__ void normal(int j, float mean, float rstd, f2* f) const {
    in.expand(j, f);
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = mul2(add2(f[e], splat(-mean)), splat(rstd));
  }
};
template <typename T, int TPR, int CH>
struct KeptRow<T, TPR, CH, true, true> {
  uint2 raw[CH];
  float scale[CH];
  const int8_t* p;
  const float* q;
  int64_t step, qstep;
  __device__ __forceinline__ KeptRow(const BackwardArgs& A, int64_t first, int64_t rows)
      : p(A.codes + first * A.cols), q(A.scales + first * A.blocks), step(rows * A.cols), qstep(rows * A.blocks) {}
  __device__ __forceinline__ void load(int t, int cols) {
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int c = Columns<TPR, true>::at(t, j, 0);
      raw[j] = c < cols ? __ldg(reinterpret_cast<const uint2*>(p + c)) : make_uint2(0, 0);
      scale[j] = c < cols ? __ldg(q + c / kBlock) : 0.0f;
    }
    p += step;
    q += qstep;
  }
  __device__ __forceinline__ void normal(int j, float mean, float rstd, f2* f) const {
    const uint32_t lo = raw[j].x ^ 0x80808080u, hi = raw[j].y ^ 0x80808080u;
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = normal_of_codes<T>(codes_f(e < 2 ? lo : hi, 2 * (e & 1)), scale[j], mean, rstd);
  }
};
template <typename T, int TPR, int CH>
struct KeptRow<T, TPR, CH, false, true> {
  int8_t raw[CH][8];
  float scale[CH][4];
  const int8_t* p;
  const float* q;
  int64_t step, qstep;
  __device__ __forceinline__ KeptRow(const BackwardArgs& A, int64_t first, int64_t rows)
      : p(A.codes + first * A.cols), q(A.scales + first * A.blocks), step(rows * A.cols), qstep(rows * A.blocks) {}
  __device__ __forceinline__ void load(int t, int cols) {
#pragma unroll
    for (int j = 0; j < CH; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = Columns<TPR, false>::at(t, j, e);
        raw[j][e] = c < cols ? p[c] : (int8_t)0;
        if ((e & 1) == 0) scale[j][e / 2] = c < cols ? q[c / kBlock] : 0.0f;
      }
    p += step;
    q += qstep;
  }
  __device__ __forceinline__ void normal(int j, float mean, float rstd, f2* f) const {
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = normal_of_codes<T>(pair((float)raw[j][2 * e], (float)raw[j][2 * e + 1]), scale[j][e], mean, rstd);
  }
};

// dx of every row, and this block's share of dgamma and dbeta.  Each thread adds up its own columns over
// the rows that it meets; at the end the block's row groups are joined in shared memory, in a fixed order.  16384 x 1024
// bf16 from the checkpoint with `add`: 26.7 us with the sums of the parts behind it, 118 MB at 4.4 TB/s; 49% of the issue
// slots, 16 warps an SM by their registers.  Four warps to a row were bound by issue (on one earlier build 29.6 us, 62%
// of the slots, where two warps took 27.6).  Single elements wait for their loads: 4099 x 1155 fp32 13.6 us (on one earlier
// build 21.1 with gamma read for every row, 16.2 with gamma in registers).
template <typename T, int TPR, int CH, bool VEC, bool CODES, bool ADD>
__global__ void __launch_bounds__(kBackThreads<TPR, CH>, kBackRoom<CH> / kBackThreads<TPR, CH>) k_ln_backward(const BackwardArgs A) {
  in_turn();
  constexpr int kGroups = kBackGroups<TPR, CH>;
  const int cols = A.cols;
  using Col = Columns<TPR, VEC>;
  __shared__ float red[kGroups][2][2 * 32];
  constexpr int kSums = 2 * CH * 4;  // pairs of sums a thread
  __shared__ f2 join[kGroups == 1 ? 1 : kGroups / 2 * kSums * TPR];
  const int t = threadIdx.x % TPR, group = threadIdx.x / TPR;
  const int64_t first = (int64_t)group * gridDim.x + blockIdx.x, step = (int64_t)gridDim.x * kGroups;
  int turn = 0;
  f2 dg[CH][4], db[CH][4];
#pragma unroll
  for (int j = 0; j < CH; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) dg[j][e] = db[j][e] = 0;
  KeptRow<T, TPR, CH, VEC, CODES> kept(A, first, step);
  RowInput<T, TPR, CH, VEC> dyin, addin;
  const T *pdy = static_cast<const T*>(A.dy) + first * A.lddy, *padd = static_cast<const T*>(A.add) + (ADD ? first * A.ldadd : 0);
  T* pdx = static_cast<T*>(A.dx) + first * A.lddx;
  float mu = 0.0f, rs = 0.0f;
  auto load = [&](int64_t r) {
    kept.load(t, cols);
    dyin.load(pdy, t, cols);
    pdy += step * A.lddy;
    mu = __ldg(A.mean + r);
    rs = __ldg(A.rstd + r);
  };
  if (first < A.rows) load(first);
  // gamma stays in registers, but beside codes and `add` only in the wide form of one group (16384 x 1155 bf16: held
  // 69.5 us, read for every row 52.0; 16384 x 1024 30.4 and 27.5)
  constexpr bool kHold = !ADD || !CODES || (VEC && CH == 1);
  f2 held[kHold ? CH : 1][4];
  if (kHold) {
#pragma unroll
    for (int j = 0; j < CH; ++j) param_group<TPR, VEC>(A.gamma, t, j, cols, held[kHold ? j : 0]);
  }
  for (int64_t r = first; r < A.rows; r += step) {
    f2 xh[CH][4], d[CH][4], s0 = 0, s1 = 0;
    const float mean = mu, rstd = rs;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      kept.normal(j, mean, rstd, xh[j]);
      dyin.expand(j, d[j]);
    }
    if (ADD) {  // needed last: this row's, not ahead
      addin.load(padd, t, cols);
      padd += step * A.ldadd;
    }
    if (r + step < A.rows) load(r + step);  // under this row's work
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      f2 gamma[4];
      if (kHold) {
#pragma unroll
        for (int e = 0; e < 4; ++e) gamma[e] = held[kHold ? j : 0][e];
      } else {
        param_group<TPR, VEC>(A.gamma, t, j, cols, gamma);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // columns past the end have dy = gamma = 0 and add nothing
        dg[j][e] = fma2(d[j][e], xh[j][e], dg[j][e]);
        db[j][e] = add2(db[j][e], d[j][e]);
        d[j][e] = mul2(d[j][e], gamma[e]);
        s0 = add2(s0, d[j][e]);
        s1 = fma2(d[j][e], xh[j][e], s1);
      }
    }
    float s[2] = {sum_of(s0), sum_of(s1)};
    row_sums<TPR>(s, red[group], turn, 1 + group);
    const f2 c0 = splat(-s[0] * A.inv_cols * rstd), c1 = splat(-s[1] * A.inv_cols * rstd);
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      f2 o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = fma2(xh[j][e], c1, fma2(d[j][e], splat(rstd), c0));
      if (ADD) {
        f2 a[4];
        addin.expand(j, a);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = add2(o[e], a[e]);
      }
      store_group<T, TPR, VEC>(pdx, t, j, cols, o);
    }
    pdx += step * A.lddx;
  }
  // the upper half of the row groups that had rows hand their sums to the lower
  const int64_t met = (A.rows - blockIdx.x + gridDim.x - 1) / gridDim.x;
  for (int n = met < kGroups ? (int)met : kGroups; n > 1; n = (n + 1) / 2) {
    const int low = (n + 1) / 2;
    f2* const to = join + (group - low) * kSums * TPR + t;
    const f2* const from = join + group * kSums * TPR + t;
    __syncthreads();
    if (group >= low && group < n) {
#pragma unroll
      for (int j = 0; j < CH; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) to[(j * 4 + e) * TPR] = dg[j][e], to[(CH * 4 + j * 4 + e) * TPR] = db[j][e];
    }
    __syncthreads();
    if (group + low < n) {
#pragma unroll
      for (int j = 0; j < CH; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          dg[j][e] = add2(dg[j][e], from[(j * 4 + e) * TPR]), db[j][e] = add2(db[j][e], from[(CH * 4 + j * 4 + e) * TPR]);
    }
  }
  if (group == 0) {
    float* p = A.part + (int64_t)blockIdx.x * 2 * cols;
#pragma unroll
    for (int j = 0; j < CH; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = Col::at(t, j, 2 * e), c1 = Col::at(t, j, 2 * e + 1);
        const float2 g = halves(dg[j][e]), b = halves(db[j][e]);
        if (c < cols) p[c] = g.x, p[cols + c] = b.x;
        if (c1 < cols) p[c1] = g.y, p[cols + c1] = b.y;
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
  in_turn();
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
    const float rstd = halves(rsqrt_rounded(splat(fmaf(block_sum(s, red), A.inv_cols, A.eps)))).x;
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
  in_turn();
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
  in_turn();
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

// the widest row of the forward and backward forms that hold rows in registers; wider ones are read again for each step
// (backward of 4096 x 8192 bf16 52 us, of 4096 x 8200 143)
constexpr int kForwardCols = 512 * 4 * 8, kBackwardCols = 512 * 2 * 8;

template <typename T, bool VEC>
cudaError_t launch_forward(const ForwardArgs& a, cudaStream_t s) {
  auto go = [&](auto tpr, auto ch, auto nr, int per_sm) {
    constexpr int kTpr = decltype(tpr)::value, kCh = decltype(ch)::value, kNr = decltype(nr)::value, kThreads = kForwardThreads<kTpr>;
    const unsigned grid = at_most(ceil_div(a.rows, kThreads / kTpr * kNr), per_sm);
    if (VEC && a.cols == kTpr * kCh * 8) return launch_after(k_ln_forward<T, kTpr, kCh, kNr, VEC, VEC>, grid, kThreads, s, a);  // no bounds to test
    return launch_after(k_ln_forward<T, kTpr, kCh, kNr, VEC, false>, grid, kThreads, s, a);
  };
  using std::integral_constant;
  using One = integral_constant<int, 1>;
  using Two = integral_constant<int, 2>;
  using Four = integral_constant<int, 4>;
  constexpr bool kLean = VEC && sizeof(T) == 2;
  // Single elements and fp32 need more registers a column: up to 2048 (wide fp32: 1024) columns a thread has eight and
  // a row the fewest warps that hold it (4099 x 1155 fp32 by single elements: 9.6 us with 160 threads, 19.8 with 128 and
  // sixteen columns each; 16384 x 1024 wide fp32: 23.9 with 128, 28.1 with a warp, but 8192 x 2048 28.5 and 24.5).
  // A warp has a 16-bit row of up to 512 columns, at 128 registers a thread (16384 x 512 6.5 us; at 96, where it spills,
  // 7.2; one row at a time 8.0; two warps a row 9.7).
  auto up_to_2048 = [&] {
    if constexpr (kLean) {
      if (a.cols <= 512) return go(integral_constant<int, 32>{}, Two{}, Two{}, 4);
      if (a.cols <= 768) return go(integral_constant<int, 96>{}, One{}, Two{}, 10);
      if (a.cols <= 1024) return go(integral_constant<int, 128>{}, One{}, Two{}, 8);
    } else {
      if (a.cols <= 512) return go(integral_constant<int, 64>{}, One{}, Two{}, 5);
      if (a.cols <= 1024) return go(integral_constant<int, 128>{}, One{}, Two{}, 5);
    }
    if constexpr (VEC) {
      return go(integral_constant<int, 128>{}, Two{}, Two{}, 5);
    } else {
      if (a.cols <= 1280) return go(integral_constant<int, 160>{}, One{}, Two{}, 4);
      if (a.cols <= 1536) return go(integral_constant<int, 192>{}, One{}, Two{}, 3);
      return go(integral_constant<int, 256>{}, One{}, Two{}, 2);
    }
  };
  if (a.cols <= 256) return go(integral_constant<int, 32>{}, One{}, Two{}, 5);
  if (a.cols <= 2048) return up_to_2048();
  if (a.cols <= 4096) return go(integral_constant<int, 256>{}, Two{}, Two{}, 2);
  // (8192 x 8192 bf16: 54 us, with 512 threads and half the columns each 73, in the form of 16384 columns 81)
  if (a.cols <= 8192) return go(integral_constant<int, 256>{}, Four{}, One{}, 2);
  if (a.cols <= kForwardCols) return go(integral_constant<int, 512>{}, Four{}, One{}, 1);
  return launch_after(k_ln_forward_wide<T>, at_most(a.rows, 8), kLnThreads, s, a);
}

// The backward form for a width: threads a row, groups of eight columns a thread.  In 16 bits, read wide, a row of
// more than 512 columns has few threads with two groups each (whole calls on one build, from x: 16384 x 1024 bf16 24.6 us,
// 27.4 with one; x 512 18.7 and 16.8); single elements and fp32 need more registers a column, so there a thread has one
// group and a row the fewest warps that hold it (16384 x 1024 fp32 with two groups a thread spilled; 4099 x 1155 fp32
// by single elements 20.8 us with 160 threads a row, 23.3 with 256).
template <typename T, bool VEC>
constexpr bool kTwoGroups = VEC && sizeof(T) == 2;
template <bool TWO, typename F>
auto with_backward_form(int64_t cols, F&& f) {
  using std::integral_constant;
  using One = integral_constant<int, 1>;
  using Two = integral_constant<int, 2>;
  if (cols <= 256) return f(integral_constant<int, 32>{}, One{});
  if (cols <= 512) return f(integral_constant<int, 64>{}, One{});
  if constexpr (TWO) {
    if (cols <= 1024) return f(integral_constant<int, 64>{}, Two{});
    if (cols <= 2048) return f(integral_constant<int, 128>{}, Two{});
    if (cols <= 4096) return f(integral_constant<int, 256>{}, Two{});
  } else {
    if (cols <= 1024) return f(integral_constant<int, 128>{}, One{});
    if (cols <= 1280) return f(integral_constant<int, 160>{}, One{});
    if (cols <= 1536) return f(integral_constant<int, 192>{}, One{});
    if (cols <= 2048) return f(integral_constant<int, 256>{}, One{});
    if (cols <= 384 * 8) return f(integral_constant<int, 384>{}, One{});
    if (cols <= 4096) return f(integral_constant<int, 512>{}, One{});
  }
  return f(integral_constant<int, 512>{}, Two{});
}
// Blocks of the backward kernel, which are the parts that the parameters' gradients are summed from.
template <bool TWO>
int backward_parts(int64_t rows, int64_t cols) {
  if (rows == 0) return 0;
  if (cols > kBackwardCols) return (int)ceil_div(rows, ceil_div(rows, 64));
  return with_backward_form<TWO>(cols, [&](auto tpr, auto ch) {
    constexpr int kCh = decltype(ch)::value, kThreads = kBackThreads<decltype(tpr)::value, kCh>;
    return (int)at_most(rows, kBackRoom<kCh> / kThreads);
  });
}

template <typename T, bool VEC, bool CODES>
cudaError_t launch_backward(const BackwardArgs& a, int parts, cudaStream_t s) {
  return with_backward_form<kTwoGroups<T, VEC>>(a.cols, [&](auto tpr, auto ch) {
    constexpr int kTpr = decltype(tpr)::value, kCh = decltype(ch)::value;
    if (a.add) return launch_after(k_ln_backward<T, kTpr, kCh, VEC, CODES, true>, parts, kBackThreads<kTpr, kCh>, s, a);
    return launch_after(k_ln_backward<T, kTpr, kCh, VEC, CODES, false>, parts, kBackThreads<kTpr, kCh>, s, a);
  });
}

template <typename T>
cudaError_t launch_backward(const BackwardArgs& a, cudaStream_t s) {
  auto on16 = [](const void* p, int64_t ld) { return aligned(p, 16) && (ld * (int64_t)sizeof(T)) % 16 == 0; };
  const bool vec = a.cols % 8 == 0 && on16(a.dy, a.lddy) && on16(a.x, a.ldx) && on16(a.add, a.ldadd) && on16(a.dx, a.lddx) && aligned(a.codes, 8) &&
                   aligned(a.gamma, 16);
  const int parts = vec ? backward_parts<kTwoGroups<T, true>>(a.rows, a.cols) : backward_parts<false>(a.rows, a.cols);
  cudaError_t e = cudaSuccess;
  if (parts == 0) {  // no rows
  } else if (a.cols > kBackwardCols) {
    e = launch_after(k_ln_backward_wide<T>, at_most(a.rows, 8), kLnThreads, s, a);
    if (e == cudaSuccess)
      e = launch_after(k_ln_param_wide<T>, dim3((unsigned)ceil_div(a.cols, kLnThreads), (unsigned)parts), kLnThreads, s, a, ceil_div(a.rows, 64));
  } else if (vec) {
    e = a.codes ? launch_backward<T, true, true>(a, parts, s) : launch_backward<T, true, false>(a, parts, s);
  } else {
    e = a.codes ? launch_backward<T, false, true>(a, parts, s) : launch_backward<T, false, false>(a, parts, s);
  }
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
  const bool vec = cols % 8 == 0 && aligned(x, 16) && aligned(y, 16) && (ldx * e) % 16 == 0 && (ldy * e) % 16 == 0 && aligned(codes, 8) &&
                   aligned(gamma, 16) && aligned(beta, 16);
  auto go = [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    return vec ? launch_forward<T, true>(a, s) : launch_forward<T, false>(a, s);
  };
  const cudaError_t ce = dtype == ONEBIT_F32 ? go((float*)nullptr) : dtype == ONEBIT_F16 ? go((__half*)nullptr) : go((__nv_bfloat16*)nullptr);
  return ce == cudaSuccess ? ONEBIT_OK : cuda_fail(ce, "onebit_layer_norm_forward");
}

extern "C" onebit_status_t onebit_layer_norm_backward_workspace(int64_t rows, int64_t cols, size_t* bytes) {
  if (!bytes) return fail(ONEBIT_ERR_INVALID_ARG, "bytes is NULL");
  onebit_status_t st = shape_ok(rows, cols);
  if (st != ONEBIT_OK) return st;
  const int a = backward_parts<false>(rows, cols), b = backward_parts<true>(rows, cols);
  *bytes = (size_t)((int64_t)(a > b ? a : b) * 2 * cols * 4);
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
