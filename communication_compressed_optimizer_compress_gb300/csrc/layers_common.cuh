// layers_common.cuh -- what the layer operators share: element types, activations, the 8-bit
// checkpoint's rounding, and the host-side argument checks.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include <initializer_list>

#include "../../include/onebit_layers.h"

namespace onebit {
namespace layers {

constexpr int kBlock = ONEBIT_CHECKPOINT_BLOCK;

// ------------------------------------------------------------------------------------------------
// element types
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// ------------------------------------------------------------------------------------------------
// activations and their derivatives, fp32
__device__ __forceinline__ float act_value(int act, float z) {
  switch (act) {
    case ONEBIT_ACT_RELU: return z > 0.0f ? z : (z != z ? z : 0.0f);
    case ONEBIT_ACT_GELU: return 0.5f * z * (1.0f + erff(z * 0.70710678f));
    case ONEBIT_ACT_GELU_TANH: return 0.5f * z * (1.0f + tanhf(0.79788456f * fmaf(0.044715f * z * z, z, z)));
    default: return z;
  }
}
__device__ __forceinline__ float act_slope(int act, float z) {
  switch (act) {
    case ONEBIT_ACT_RELU: return z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
    case ONEBIT_ACT_GELU:
      return fmaf(z * 0.39894228f, expf(-0.5f * z * z), 0.5f * (1.0f + erff(z * 0.70710678f)));
    case ONEBIT_ACT_GELU_TANH: {
      const float t = tanhf(0.79788456f * fmaf(0.044715f * z * z, z, z));
      return fmaf(0.5f * z * (1.0f - t * t), 0.79788456f * fmaf(0.134145f * z, z, 1.0f), 0.5f * (1.0f + t));
    }
    default: return 1.0f;
  }
}

// ------------------------------------------------------------------------------------------------
// the 8-bit checkpoint's rounding.  `most` is the block's largest |x| (NaN or infinite if the block
// holds such a value).
struct BlockScale {
  float scale;  // what a code is multiplied by
  float inv;    // what a value is multiplied by before it is rounded to a code
};
__device__ __forceinline__ BlockScale block_scale(float most) {
  if (!(most <= 3.4028234663852886e38f)) return {CUDART_NAN_F, 0.0f};
  if (most < 7.52316384526264e-37f) return {0.0f, 0.0f};  // 2^-120: 127/most stays finite above it
  return {__fdiv_rn(most, 127.0f), __fdiv_rn(127.0f, most)};
}
// code of one value, in the low byte: adding 1.5*2^23 leaves the nearest integer (ties to even) in
// the low bits of the sum.  A block with inv = 0 that holds inf or NaN (inf*0) gets code 0.
__device__ __forceinline__ uint32_t code_of(float x, float inv) {
  return inv == 0.0f ? 0u : (__float_as_uint(__fadd_rn(__fmul_rn(x, inv), 12582912.0f)) & 0xffu);
}
// what a code stands for.  The scale is a/127 rounded, so that 127 times it can round past the largest
// fp32 value when a is (almost) that value: such a product is a itself.  Only an fp32 matrix holds such.
template <typename T>
__device__ __forceinline__ float value_of(int code, float scale) {
  const float v = __fmul_rn((float)code, scale);
  return sizeof(T) == 4 && isinf(v) ? copysignf(3.4028234663852886e38f, v) : v;
}
// the larger of two magnitudes, NaN if either is NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// ------------------------------------------------------------------------------------------------
// warp sums (every lane gets the total, the same order in each)
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max_nan(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// ------------------------------------------------------------------------------------------------
// host side

// Records a message for onebit_layers_last_error() and returns the status.
onebit_status_t fail(onebit_status_t status, const char* what);
onebit_status_t cuda_fail(cudaError_t e, const char* where);
int sm_count();  // of the current device

inline int dtype_size(int32_t dtype) { return dtype == ONEBIT_F32 ? 4 : 2; }
inline bool dtype_ok(int32_t dtype) { return dtype >= ONEBIT_F32 && dtype <= ONEBIT_BF16; }

struct Span {
  const char* p;
  int64_t bytes;
};
inline Span span_of(const void* p, int64_t bytes) { return Span{static_cast<const char*>(p), p ? bytes : 0}; }
inline Span matrix(const void* p, int64_t rows, int64_t ld, int64_t cols, int64_t size) {
  return span_of(p, rows > 0 ? ((rows - 1) * ld + cols) * size : 0);
}
inline bool overlap(const Span& a, const Span& b) {
  return a.bytes > 0 && b.bytes > 0 && a.p < b.p + b.bytes && b.p < a.p + a.bytes;
}
// every output disjoint from every input and from the other outputs
inline bool disjoint(std::initializer_list<Span> in, std::initializer_list<Span> out) {
  for (const Span* o = out.begin(); o != out.end(); ++o) {
    for (const Span& i : in)
      if (overlap(*o, i)) return false;
    for (const Span* q = out.begin(); q != o; ++q)
      if (overlap(*o, *q)) return false;
  }
  return true;
}
inline bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Widths and row counts beyond these have no use on one device; within them every element offset
// fits 63 bits and every tile index 31.
constexpr int64_t kMaxRows = (int64_t)1 << 31;
constexpr int64_t kMaxCols = (int64_t)1 << 24;

}  // namespace layers
}  // namespace onebit
