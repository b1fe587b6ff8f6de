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
// Activations and their derivatives, fp32.
//
// Phi(z), the normal distribution function, by Hastings' rational approximation (Abramowitz and Stegun
// 7.1.26): with a = |z| and t = 1/(1 + 0.3275911 a/sqrt(2)), 1 - Phi(a) = t (c1 + t (c2 + t (c3 + t (c4 +
// t c5)))) exp(-a^2/2) to 7.5e-8.  It needs the exponential that the derivative needs too, one reciprocal
// and no branch: 16 instructions for gelu, 21 for gelu and its derivative together (the library's erff and
// expf: 47).  Beyond |z| = 40 the tail is 0 in fp32; the clamp there keeps infinities from meeting zeros,
// and passes NaN on.
//
// The tanh form is z times the logistic function of 2 sqrt(2/pi) (z + 0.044715 z^3).
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// the larger of two values, NaN if either is NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
struct ActPair {
  float value, slope;
};
template <int ACT, bool VALUE, bool SLOPE>
__device__ __forceinline__ ActPair act_pair(float z) {
  ActPair p{z, 1.0f};
  if (ACT == ONEBIT_ACT_RELU) {
    if (VALUE) p.value = max_nan(z, 0.0f);
    if (SLOPE) p.slope = z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
  } else if (ACT == ONEBIT_ACT_GELU) {
    const float a = min_nan(fabsf(z), 40.0f);
    const float e = exp2_fast(a * a * -0.72134752f);  // -1/(2 ln 2)
    const float t = rcp_fast(fmaf(a, 0.23164190f, 1.0f));
    float q = fmaf(t, 0.53070271f, -0.72657601f);
    q = fmaf(t, q, 0.71070687f);
    q = fmaf(t, q, -0.14224837f);
    q = fmaf(t, q, 0.12741480f);
    const float tail = q * t * e;
    if (VALUE) p.value = fmaf(-a, tail, fmaxf(z, 0.0f));
    if (SLOPE) p.slope = 0.5f + copysignf(fmaf(a * 0.39894228f, e, 0.5f - tail), z);
  } else if (ACT == ONEBIT_ACT_GELU_TANH) {
    const float c = SLOPE ? min_nan(max_nan(z, -40.0f), 40.0f) : max_nan(z, -40.0f);
    const float zz = c * c;
    // -2 sqrt(2/pi) / ln 2 = -2.3022082
    const float s = rcp_fast(1.0f + exp2_fast(c * fmaf(zz, -0.10294324f, -2.3022082f)));
    if (VALUE) p.value = (SLOPE ? max_nan(z, -40.0f) : c) * s;
    if (SLOPE) p.slope = fmaf(c * s * (1.0f - s), fmaf(zz, 0.21406445f, 1.5957691f), s);
  }
  return p;
}
template <int ACT>
__device__ __forceinline__ float act_value(float z) { return act_pair<ACT, true, false>(z).value; }
template <int ACT>
__device__ __forceinline__ float act_slope(float z) { return act_pair<ACT, false, true>(z).slope; }
__device__ __forceinline__ float act_value(int act, float z) {
  return act == ONEBIT_ACT_GELU ? act_value<ONEBIT_ACT_GELU>(z)
         : act == ONEBIT_ACT_RELU ? act_value<ONEBIT_ACT_RELU>(z)
         : act == ONEBIT_ACT_GELU_TANH ? act_value<ONEBIT_ACT_GELU_TANH>(z) : z;
}
__device__ __forceinline__ float act_slope(int act, float z) {
  return act == ONEBIT_ACT_GELU ? act_slope<ONEBIT_ACT_GELU>(z)
         : act == ONEBIT_ACT_RELU ? act_slope<ONEBIT_ACT_RELU>(z)
         : act == ONEBIT_ACT_GELU_TANH ? act_slope<ONEBIT_ACT_GELU_TANH>(z) : 1.0f;
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
// A code as fp32, exactly: the byte, made unsigned, becomes the low bits of 2^23, from which 2^23 + 128
// is taken away (a byte permute and an addition; the conversion unit does a quarter as many).
__device__ __forceinline__ float code_f(uint32_t biased_word, int byte) {
  return __uint_as_float(__byte_perm(biased_word, 0x4b000000u, 0x7650 + byte)) - 8388736.0f;
}
// four codes of a word, which the caller has XORed with 0x80808080
template <typename T>
__device__ __forceinline__ void values4(uint32_t word, float scale, float* v) {
  word ^= 0x80808080u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = __fmul_rn(code_f(word, i), scale);
    if (sizeof(T) == 4 && isinf(v[i])) v[i] = copysignf(3.4028234663852886e38f, v[i]);
  }
}
// four values to a word of codes; inv is 0 only for blocks whose codes are all 0
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float inv) {
  const uint32_t x = __float_as_uint(__fadd_rn(__fmul_rn(a, inv), 12582912.0f)), y = __float_as_uint(__fadd_rn(__fmul_rn(b, inv), 12582912.0f));
  const uint32_t z = __float_as_uint(__fadd_rn(__fmul_rn(c, inv), 12582912.0f)), w = __float_as_uint(__fadd_rn(__fmul_rn(d, inv), 12582912.0f));
  const uint32_t r = __byte_perm(__byte_perm(x, y, 0x0040), __byte_perm(z, w, 0x0040), 0x5410);
  return inv == 0.0f ? 0u : r;  // inf and NaN times 0 would leave other bits
}

// ------------------------------------------------------------------------------------------------
// eight elements at once: 16 bytes of a 16-bit type, 32 of fp32
template <typename T>
struct Raw8 {
  uint4 v[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Raw8<T> load8(const T* p) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.v[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  return r;
}
__device__ __forceinline__ void expand8(const Raw8<float>& r, float* f) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    f[4 * i] = __uint_as_float(r.v[i].x), f[4 * i + 1] = __uint_as_float(r.v[i].y);
    f[4 * i + 2] = __uint_as_float(r.v[i].z), f[4 * i + 3] = __uint_as_float(r.v[i].w);
  }
}
__device__ __forceinline__ void expand8(const Raw8<__half>& r, float* f) {
  const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    f[2 * i] = h.x, f[2 * i + 1] = h.y;
  }
}
__device__ __forceinline__ void expand8(const Raw8<__nv_bfloat16>& r, float* f) {
  const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[2 * i] = __uint_as_float(w[i] << 16), f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void store8(float* p, const float* f) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float* f) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]), pack2<T>(f[4], f[5]), pack2<T>(f[6], f[7]));
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
// Kernels of one call follow each other with programmatic launches: the next kernel's blocks may start
// when every block of the one before has started (and there is room), and wait where they need its
// results.  A kernel that does not need them still waits before it ends, so that the end of a call's last
// kernel is the end of them all.
__device__ __forceinline__ void launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Sums of `parts` partial rows of `width` fp32 columns, in a fixed order; columns below `split` go to lo,
// the others to hi.  A block has 32 columns, 32 threads to each.
constexpr int kSumRows = 32;
template <typename G>
static __global__ void __launch_bounds__(32 * kSumRows) k_sum_parts(const float* __restrict__ part, int64_t parts, int64_t width, int64_t split,
                                                                    G* __restrict__ lo, G* __restrict__ hi) {
  __shared__ float red[kSumRows][33];
  const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  wait_previous();
  float s = 0.0f;
  if (c < width) {
#pragma unroll 8
    for (int64_t p = row; p < parts; p += kSumRows) s += part[p * width + c];
  }
  red[row][lane] = s;
  __syncthreads();
  const float t = warp_sum(red[lane][row]);  // column `row` of the block's 32
  const int64_t o = (int64_t)blockIdx.x * 32 + row;
  if (lane == 0 && o < width) {
    if (o < split) lo[o] = from_f<G>(t);
    else hi[o - split] = from_f<G>(t);
  }
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

template <typename... Params, typename... Args>
inline cudaError_t launch_after(void (*kernel)(Params...), dim3 grid, int threads, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}
template <typename G>
inline cudaError_t sum_parts(const float* part, int64_t parts, int64_t width, int64_t split, void* lo, void* hi, cudaStream_t s) {
  return launch_after(k_sum_parts<G>, dim3((unsigned)ceil_div(width, 32)), 32 * kSumRows, s, part, parts, width, split, static_cast<G*>(lo),
                      static_cast<G*>(hi));
}
inline cudaError_t sum_parts(int32_t dtype, const float* part, int64_t parts, int64_t width, int64_t split, void* lo, void* hi, cudaStream_t s) {
  return dtype == ONEBIT_F32   ? sum_parts<float>(part, parts, width, split, lo, hi, s)
         : dtype == ONEBIT_F16 ? sum_parts<__half>(part, parts, width, split, lo, hi, s)
                               : sum_parts<__nv_bfloat16>(part, parts, width, split, lo, hi, s);
}

// Widths and row counts beyond these have no use on one device; within them every element offset
// fits 63 bits and every tile index 31.
constexpr int64_t kMaxRows = (int64_t)1 << 31;
constexpr int64_t kMaxCols = (int64_t)1 << 24;

}  // namespace layers
}  // namespace onebit
