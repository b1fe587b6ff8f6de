// linear_common.cuh -- what the linear layer's forward and backward pass share: realigned copies of
// operands, epilogues over the partial sums of a cut contraction, workspace layout.
#pragma once

#include "tensor_product.cuh"

namespace onebit {
namespace layers {

inline int64_t pad256(int64_t b) { return (b + 255) & ~(int64_t)255; }
inline int64_t pad8(int64_t c) { return (c + 7) & ~(int64_t)7; }

// Can TMA read this matrix as it lies?  (16-byte base, row stride a multiple of 16 bytes)
inline bool copyable(const void* p, int64_t ld) { return aligned(p, 16) && ld % 8 == 0; }
inline bool vec16(const void* p, int64_t ld) { return aligned(p, 16) && ld % 8 == 0; }

template <typename T>
inline Input16<T> make_input(const void* p, int64_t ld) {
  return {static_cast<const T*>(p), ld, aligned(p, 32) && ld % 16 == 0, vec16(p, ld)};
}

inline unsigned flat_grid(int64_t total, int threads) {
  const int64_t most = (int64_t)sm_count() * 8, want = ceil_div(total, threads);
  return (unsigned)(want < most ? want : most);
}

// Hands out pieces of the caller's workspace; with a NULL base it only adds them up.
struct Space {
  char* base;
  int64_t used = 0;
  template <typename T>
  T* take(int64_t count) {
    char* p = base ? base + used : nullptr;
    used += pad256(count * (int64_t)sizeof(T));
    return reinterpret_cast<T*>(p);
  }
};

// Rows of any alignment into rows of ld = pad8(cols) on 16 bytes (the columns past the end are not read).  Up to
// three matrices in one launch, one to each blockIdx.y.  Inside a row by whole words, shifted where the columns lie across
// them (linear of 4144 x 3136 x 416 in odd rows 24.8 us, 28.8 by single elements).  Latency of a launch for small
// matrices: 3 us for 1237 x 1001 and 777 x 1001.
struct Realign {
  const uint16_t* x;
  int64_t ldx, rows, ld;
  int cols;
  uint16_t* out;
};
struct Realigns {
  Realign m[3];
};
static __global__ void __launch_bounds__(256) k_realign(const Realigns all) {
  in_turn();
  const Realign& a = all.m[blockIdx.y];
  const int64_t per = a.ld / 8, total = a.rows * per;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / per;
    const int c = (int)(i - r * per) * 8;
    uint32_t v[4];
    const uint16_t* const x = a.x + r * a.ldx + c;
    if (c > 0 && c + 8 < a.cols) {  // whole words, which hold columns c - 1 to c + 8 where the columns lie across them
      const bool across = reinterpret_cast<uintptr_t>(x) & 2;
      const uint32_t* const w = reinterpret_cast<const uint32_t*>(x - across);
      uint32_t t[5];
#pragma unroll
      for (int q = 0; q < 4; ++q) t[q] = w[q];
      t[4] = across ? w[4] : 0;
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = across ? __funnelshift_r(t[q], t[q + 1], 16) : t[q];
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t lo = c + 2 * q < a.cols ? x[2 * q] : 0, hi = c + 2 * q + 1 < a.cols ? x[2 * q + 1] : 0;
        v[q] = lo | hi << 16;
      }
    }
    *reinterpret_cast<uint4*>(a.out + r * a.ld + c) = make_uint4(v[0], v[1], v[2], v[3]);
  }
}

// The operands as TMA can read them: themselves, or realigned copies in the workspace, made by run().
struct Readable {
  Realigns all{};
  int n = 0;
  int64_t most = 0;
  Operand take(Space& ws, const void* p, int64_t ld, int64_t rows, int64_t cols) {
    if (copyable(p, ld)) return {p, ld};
    const int64_t ldc = pad8(cols);
    uint16_t* c = ws.take<uint16_t>(rows * ldc);
    all.m[n++] = Realign{static_cast<const uint16_t*>(p), ld, rows, ldc, (int)cols, c};
    if (rows * ldc / 8 > most) most = rows * ldc / 8;
    return {c, ldc};
  }
  cudaError_t run(cudaStream_t s) const {
    return n == 0 ? cudaSuccess : launch_after(k_realign, dim3(flat_grid(most, 256), (unsigned)n), 256, s, all);
  }
};

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

// The partial products of a cut contraction: splits x rows x ld in fp32, added in order.
struct Partials {
  const float* p;
  int64_t ld, split_stride;
  int splits;
  __device__ __forceinline__ float at(int64_t r, int c) const {
    float s = p[r * ld + c];
    for (int i = 1; i < splits; ++i) s += p[i * split_stride + r * ld + c];
    return s;
  }
  // columns c to c + 3, c a multiple of 4 (a row's end is padded to that)
  __device__ __forceinline__ void at4(int64_t r, int c, float (&s)[4]) const {
    const float* q = p + r * ld + c;
    float4 t = *reinterpret_cast<const float4*>(q);
#pragma unroll 4
    for (int i = 1; i < splits; ++i) {
      const float4 u = *reinterpret_cast<const float4*>(q + i * split_stride);
      t.x += u.x, t.y += u.y, t.z += u.z, t.w += u.w;
    }
    s[0] = t.x, s[1] = t.y, s[2] = t.z, s[3] = t.w;
  }
};
inline Partials take_partials(Space& ws, const ProductPlan& plan, int64_t rows, int64_t cols) {
  Partials q{};
  if (plan.splits == 1) return q;
  q.ld = (cols + 3) & ~(int64_t)3;
  q.split_stride = ((rows + 31) & ~(int64_t)31) * q.ld;
  q.splits = plan.splits;
  q.p = ws.take<float>(q.split_stride * plan.splits);
  return q;
}
// Each split's tile rows are a multiple of the store boxes' (32): a box never reaches into the next split.
inline cudaError_t to_partials(PlainEpilogue<float>* e, const Partials& q, int64_t cols) {
  e->split_rows = q.split_stride / q.ld;
  return make_output(&e->out, const_cast<float*>(q.p), e->split_rows * q.splits, cols, q.ld);
}

template <typename F>
void with_grad(int32_t dtype, void* p, F&& f) {
  if (dtype == ONEBIT_F32) f(static_cast<float*>(p));
  else if (dtype == ONEBIT_F16) f(static_cast<__half*>(p));
  else f(static_cast<__nv_bfloat16*>(p));
}

inline onebit_status_t linear_shape_ok(int64_t rows, int64_t in, int64_t out, int32_t dtype, int32_t act) {
  if (rows < 0 || in < 1 || out < 1) return fail(ONEBIT_ERR_INVALID_ARG, "rows or widths out of range");
  if (rows > kMaxRows || in > kMaxCols || out > kMaxCols)
    return fail(ONEBIT_ERR_UNSUPPORTED, "more than 2^31 rows or a width above 2^24");
  if (!dtype_ok(dtype)) return fail(ONEBIT_ERR_INVALID_ARG, "dtype is not one of f32, f16, bf16");
  if (dtype == ONEBIT_F32) return fail(ONEBIT_ERR_UNSUPPORTED, "the linear layer takes f16 or bf16 operands");
  if (act < ONEBIT_ACT_NONE || act > ONEBIT_ACT_GELU_TANH) return fail(ONEBIT_ERR_INVALID_ARG, "unknown activation");
  return ONEBIT_OK;
}

}  // namespace layers
}  // namespace onebit
