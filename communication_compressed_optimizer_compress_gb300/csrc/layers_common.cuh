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
// Two fp32 values in a register pair: one instruction adds, multiplies or fuses both.  The streaming
// kernels and the products' epilogues are close to the issue limit, so their arithmetic goes by pairs.
using f2 = unsigned long long;
__device__ __forceinline__ f2 pair(float lo, float hi) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ f2 splat(float x) { return pair(x, x); }
__device__ __forceinline__ float2 halves(f2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float sum_of(f2 v) {
  const float2 h = halves(v);
  return h.x + h.y;
}

// the larger of two values, NaN if either is NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// the largest of m and two magnitudes, NaN if any is NaN
__device__ __forceinline__ float max_abs(float m, f2 v) {
  const float2 h = halves(v);
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(h.x), "f"(h.y));
  return r;
}
// |z| held to at most 6, and z itself to a magnitude of at most 40; NaN stays NaN
__device__ __forceinline__ float magnitude6(float z) {
  float r;
  asm("min.NaN.abs.f32 %0, %1, %2, %2;" : "=f"(r) : "f"(z), "f"(6.0f));
  return r;
}
__device__ __forceinline__ float held40(float z) {
  float r;
  asm("min.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(r) : "f"(z), "f"(40.0f));
  return r;
}
__device__ __forceinline__ float held87(float z) {
  float r;
  asm("min.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(r) : "f"(z), "f"(87.0f));
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

// ------------------------------------------------------------------------------------------------
// Activations and their derivatives, fp32, two at a time.
//
// gelu(z) = max(z, 0) - a (1 - Phi(a)), a = |z|.  log2(1 - Phi(a)) is a smooth, nearly quadratic function, so
// the tail is one exponential of a polynomial: degree 6, fitted here on [0, 6] by least squares with the
// weights of gelu's own error, raised where it was largest until it levelled out.  It leaves gelu within
// 3.8e-7 and Phi within 2e-7 in fp32, for 14 instructions a pair (a rational form with its reciprocal and
// second exponential: 22).  Beyond 6 the product a (1 - Phi(a)) is 6e-9 and stays there.  The derivative
// Phi(z) + z phi(z) = 1/2 + sign(z) (1/2 - tail + a phi(a)) needs one exponential more.
//
// The tanh form is z times the logistic function of 2 sqrt(2/pi) (z + 0.044715 z^3), silu z times that of z.  silu's
// argument is held to 87, where exp(87) and its reciprocal are still normal numbers: below -87 silu stays at -1.4e-36.
//
// The constants come as register pairs: as literals they would be set up again for each pair, which was
// a third of the instructions of the products' epilogues.
constexpr int kActConsts = 10;
struct ActConsts {
  f2 k[kActConsts];
};
__host__ __device__ constexpr float act_const(int act, int i) {
  constexpr float gelu[kActConsts] = {-0.9999995231628418f, -1.151128888130188f, -0.45901408791542053f, -0.05307028442621231f, 0.007853773422539234f,
                                      -0.0006991532281972468f, 2.503262112441007e-05f,
                                      -0.72134752f,  // -1/(2 ln 2)
                                      0.39894228f,   // 1/sqrt(2 pi)
                                      0.5f};
  // -2 sqrt(2/pi) / ln 2 times 0.044715 and 1; 2 sqrt(2/pi) times 3 * 0.044715 and 1
  constexpr float tanh[kActConsts] = {-0.10294324f, -2.3022082f, 1.0f, 0.21406445f, 1.5957691f};
  constexpr float silu[kActConsts] = {-1.4426950f, 1.0f};  // -1/ln 2
  return act == ONEBIT_ACT_GELU ? gelu[i] : act == ONEBIT_ACT_GELU_TANH ? tanh[i] : act == ONEBIT_ACT_SILU ? silu[i] : 0.0f;
}
template <int ACT>
__device__ __forceinline__ ActConsts literal_consts() {
  ActConsts c;
#pragma unroll
  for (int i = 0; i < kActConsts; ++i) c.k[i] = splat(act_const(ACT, i));
  return c;
}
template <int ACT, bool VALUE, bool SLOPE>
__device__ __forceinline__ void activate(const ActConsts& c, f2 z2, f2& value, f2& slope) {
  const f2* k = c.k;
  if (ACT == ONEBIT_ACT_NONE) {
    value = z2;
    slope = splat(1.0f);
    return;
  }
  const float2 z = halves(z2);
  if (ACT == ONEBIT_ACT_RELU) {
    if (VALUE) value = pair(max_nan(z.x, 0.0f), max_nan(z.y, 0.0f));
    if (SLOPE) slope = pair(z.x > 0.0f ? 1.0f : (z.x != z.x ? z.x : 0.0f), z.y > 0.0f ? 1.0f : (z.y != z.y ? z.y : 0.0f));
  } else if (ACT == ONEBIT_ACT_GELU) {
    const float2 a = make_float2(magnitude6(z.x), magnitude6(z.y));
    const f2 a2 = pair(a.x, a.y);
    f2 p = k[6];
#pragma unroll
    for (int i = 5; i >= 0; --i) p = fma2(p, a2, k[i]);
    const float2 l = halves(p), tail = make_float2(exp2_fast(l.x), exp2_fast(l.y));
    if (VALUE) value = pair(fmaf(-a.x, tail.x, fmaxf(z.x, 0.0f)), fmaf(-a.y, tail.y, fmaxf(z.y, 0.0f)));
    if (SLOPE) {
      const float2 g = halves(mul2(mul2(a2, a2), k[7]));
      const float2 m = halves(fma2(mul2(a2, k[8]), pair(exp2_fast(g.x), exp2_fast(g.y)), add2(k[9], pair(-tail.x, -tail.y))));
      slope = add2(pair(copysignf(m.x, z.x), copysignf(m.y, z.y)), k[9]);
    }
  } else if (ACT == ONEBIT_ACT_SILU) {
    const f2 c2 = pair(held87(z.x), held87(z.y));
    const float2 g = halves(mul2(c2, k[0]));
    const float2 u = halves(add2(pair(exp2_fast(g.x), exp2_fast(g.y)), k[1]));
    const f2 s = pair(rcp_fast(u.x), rcp_fast(u.y));
    if (VALUE) value = mul2(pair(max_nan(z.x, -87.0f), max_nan(z.y, -87.0f)), s);
    if (SLOPE) {
      const float2 h = halves(s);
      slope = fma2(mul2(c2, s), add2(k[1], pair(-h.x, -h.y)), s);
    }
  } else {
    const f2 c2 = pair(held40(z.x), held40(z.y)), zz = mul2(c2, c2);
    const float2 g = halves(mul2(c2, fma2(zz, k[0], k[1])));
    const float2 u = halves(add2(pair(exp2_fast(g.x), exp2_fast(g.y)), k[2]));
    const f2 s = pair(rcp_fast(u.x), rcp_fast(u.y));
    if (VALUE) value = mul2(pair(max_nan(z.x, -40.0f), max_nan(z.y, -40.0f)), s);
    if (SLOPE) {
      const float2 h = halves(s);
      slope = fma2(mul2(mul2(c2, s), add2(k[2], pair(-h.x, -h.y))), fma2(zz, k[3], k[4]), s);
    }
  }
}
// The same without registers for the constants, for an epilogue that has none left: literals, and gelu's ten pairs (where that is the
// form that does not spill, the tanh form's five too) as those of single operations, seven instructions a pair more.
__device__ __forceinline__ float2 gelu_single(float z) {  // value and slope
  constexpr int A = ONEBIT_ACT_GELU;
  const float a = magnitude6(z);
  float p = act_const(A, 6);
#pragma unroll
  for (int i = 5; i >= 0; --i) p = fmaf(p, a, act_const(A, i));
  const float tail = exp2_fast(p), m = fmaf(a * act_const(A, 8), exp2_fast(a * a * act_const(A, 7)), act_const(A, 9) - tail);
  return make_float2(fmaf(-a, tail, fmaxf(z, 0.0f)), copysignf(m, z) + act_const(A, 9));
}
__device__ __forceinline__ float2 gelu_tanh_single(float z) {
  constexpr int A = ONEBIT_ACT_GELU_TANH;
  const float c = held40(z), zz = c * c, s = rcp_fast(exp2_fast(c * fmaf(zz, act_const(A, 0), act_const(A, 1))) + 1.0f);
  return make_float2(max_nan(z, -40.0f) * s, fmaf(c * s * (1.0f - s), fmaf(zz, act_const(A, 3), act_const(A, 4)), s));
}
template <int ACT, bool SINGLE_TANH = false>
__device__ __forceinline__ void activate_lean(f2 z2, f2& value, f2& slope) {
  if constexpr (ACT == ONEBIT_ACT_GELU || (ACT == ONEBIT_ACT_GELU_TANH && SINGLE_TANH)) {
    const float2 z = halves(z2), lo = ACT == ONEBIT_ACT_GELU ? gelu_single(z.x) : gelu_tanh_single(z.x),
                 hi = ACT == ONEBIT_ACT_GELU ? gelu_single(z.y) : gelu_tanh_single(z.y);
    value = pair(lo.x, hi.x), slope = pair(lo.y, hi.y);
  } else {
    activate<ACT, true, true>(literal_consts<ACT>(), z2, value, slope);
  }
}
template <int ACT>
__device__ __forceinline__ f2 act2(const ActConsts& c, f2 z) {
  f2 v, s;
  activate<ACT, true, false>(c, z, v, s);
  return v;
}
// one value, for the kernels off the hot paths
template <int ACT>
__device__ __forceinline__ float2 act_one(float z) {  // value and slope
  f2 v = splat(z), s = splat(1.0f);
  activate<ACT, true, true>(literal_consts<ACT>(), splat(z), v, s);
  return make_float2(halves(v).x, halves(s).x);
}
__device__ __forceinline__ float2 act_both(int act, float z) {
  return act == ONEBIT_ACT_GELU ? act_one<ONEBIT_ACT_GELU>(z)
         : act == ONEBIT_ACT_RELU ? act_one<ONEBIT_ACT_RELU>(z)
         : act == ONEBIT_ACT_GELU_TANH ? act_one<ONEBIT_ACT_GELU_TANH>(z) : make_float2(z, 1.0f);
}
__device__ __forceinline__ float act_value(int act, float z) { return act_both(act, z).x; }
__device__ __forceinline__ float act_slope(int act, float z) { return act_both(act, z).y; }

// ------------------------------------------------------------------------------------------------
// the 8-bit checkpoint's rounding.  `most` is the block's largest |x| (NaN or infinite if the block
// holds such a value).
struct BlockScale {
  float scale;  // what a code is multiplied by
  float inv;    // what a value is multiplied by before it is rounded to a code
};
// Both quotients by one correction of an approximate one (Markstein 1990): q += r (n - d q), which leaves
// them rounded as a division would (compared for every mantissa).  A division of the language is several times as
// long, and every eight columns of a layer norm's row need two.
__device__ __forceinline__ BlockScale block_scale(float most) {
  if (!(most <= 3.4028234663852886e38f)) return {CUDART_NAN_F, 0.0f};
  if (most < 7.52316384526264e-37f) return {0.0f, 0.0f};  // 2^-120
  const float q = most * 0.0078740157f;
  const float scale = fmaf(fmaf(q, -127.0f, most), 0.0078740157f, q);
  // the reciprocal of most/4: neither it nor a factor below leaves the normal range
  const float r = rcp_fast(most * 0.25f), p = r * 31.75f;
  return {scale, fmaf(fmaf(p, -most, 127.0f) * 0.25f, r, p)};
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
// Codes as fp32, exactly: a byte, made unsigned, becomes the low bits of 2^23, from which 2^23 + 128 is
// taken away (a byte permute and half an addition; the conversion unit does a quarter as many).
__device__ __forceinline__ f2 codes_f(uint32_t biased, int byte) {  // two bytes from `byte` on, XORed with 0x80
  return add2(pair(__uint_as_float(__byte_perm(biased, 0x4b000000u, 0x7650 + byte)), __uint_as_float(__byte_perm(biased, 0x4b000000u, 0x7651 + byte))),
              splat(-8388736.0f));
}
// what the four codes of a word stand for
template <typename T>
__device__ __forceinline__ void values4(uint32_t word, float scale, f2* v) {
  word ^= 0x80808080u;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    v[i] = mul2(codes_f(word, 2 * i), splat(scale));
    if (sizeof(T) == 4) {
      float2 h = halves(v[i]);
      if (isinf(h.x)) h.x = copysignf(3.4028234663852886e38f, h.x);
      if (isinf(h.y)) h.y = copysignf(3.4028234663852886e38f, h.y);
      v[i] = pair(h.x, h.y);
    }
  }
}
// four values to a word of codes.  The product is rounded before 1.5*2^23 is added, as in code_of(): the additions go
// one by one, as a packed product and a packed sum behind it are compiled to one fused operation, whatever rounding they
// name (codes at ties then differed between the layouts).  The caller sees to inv = 0 where values may be inf or NaN.
__device__ __forceinline__ uint32_t codes4_finite(f2 ab, f2 cd, float inv) {
  const float2 p = halves(mul2(ab, splat(inv))), q = halves(mul2(cd, splat(inv)));
  const float2 x = make_float2(__fadd_rn(p.x, 12582912.0f), __fadd_rn(p.y, 12582912.0f)), y = make_float2(__fadd_rn(q.x, 12582912.0f), __fadd_rn(q.y, 12582912.0f));
  return __byte_perm(__byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x0040),
                     __byte_perm(__float_as_uint(y.x), __float_as_uint(y.y), 0x0040), 0x5410);
}
// inv is 0 only for blocks whose codes are all 0
__device__ __forceinline__ uint32_t codes4(f2 ab, f2 cd, float inv) {
  const uint32_t r = codes4_finite(ab, cd, inv);
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
// 32 bytes at once (the address lies on 32): a warp's accesses then cover whole lines
__device__ __forceinline__ void load32(const void* p, uint32_t* v) {
  asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
               : "l"(p));
}
__device__ __forceinline__ void store32(void* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]),
               "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void expand8(const Raw8<float>& r, f2* f) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    f[2 * i] = pair(__uint_as_float(r.v[i].x), __uint_as_float(r.v[i].y));
    f[2 * i + 1] = pair(__uint_as_float(r.v[i].z), __uint_as_float(r.v[i].w));
  }
}
template <typename T>
__device__ __forceinline__ f2 widen(uint32_t v);  // two 16-bit values
template <>
__device__ __forceinline__ f2 widen<__half>(uint32_t v) {
  const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&v));
  return pair(h.x, h.y);
}
template <>
__device__ __forceinline__ f2 widen<__nv_bfloat16>(uint32_t v) {
  return pair(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
template <typename T>
__device__ __forceinline__ void expand8(const Raw8<T>& r, f2* f) {
  f[0] = widen<T>(r.v[0].x), f[1] = widen<T>(r.v[0].y), f[2] = widen<T>(r.v[0].z), f[3] = widen<T>(r.v[0].w);
}
template <typename T>
__device__ __forceinline__ uint32_t narrow(f2 v);  // two values, rounded
template <>
__device__ __forceinline__ uint32_t narrow<__half>(f2 v) {
  const float2 f = halves(v);
  const __half2 h = __floats2half2_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t narrow<__nv_bfloat16>(f2 v) {
  const float2 f = halves(v);
  const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void store8(float* p, const f2* f) {
  const float2 a = halves(f[0]), b = halves(f[1]), c = halves(f[2]), d = halves(f[3]);
  *reinterpret_cast<float4*>(p) = make_float4(a.x, a.y, b.x, b.y);
  *reinterpret_cast<float4*>(p + 4) = make_float4(c.x, c.y, d.x, d.y);
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const f2* f) {
  *reinterpret_cast<uint4*>(p) = make_uint4(narrow<T>(f[0]), narrow<T>(f[1]), narrow<T>(f[2]), narrow<T>(f[3]));
}

// 16 elements on 32 bytes
template <typename T>
__device__ __forceinline__ void load16(const T* p, f2* f) {
  uint32_t v[8];
#pragma unroll
  for (int h = 0; h < (int)sizeof(T) / 2; ++h) {
    load32(p + h * (32 / sizeof(T)), v);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (sizeof(T) == 2) f[i] = widen<T>(v[i]);
      else if (i % 2 == 0) f[4 * h + i / 2] = pair(__uint_as_float(v[i]), __uint_as_float(v[i + 1]));
    }
  }
}
template <typename T>
__device__ __forceinline__ void store16(T* p, const f2* f) {
  uint32_t v[8];
#pragma unroll
  for (int h = 0; h < (int)sizeof(T) / 2; ++h) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (sizeof(T) == 2) {
        v[i] = narrow<T>(f[i]);
      } else if (i % 2 == 0) {
        const float2 x = halves(f[4 * h + i / 2]);
        v[i] = __float_as_uint(x.x), v[i + 1] = __float_as_uint(x.y);
      }
    }
    store32(p + h * (32 / sizeof(T)), v);
  }
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

// 1/sqrt(v) of two values, rounded: one Newton step on CUDA's, which is within two ulps, with what v y rounds off taken
// along (1 - v y^2 = 1 - s y + (s - v y) y).  The step of 0 and of infinity is NaN: their reciprocals are there before it.
__device__ __forceinline__ f2 rsqrt_rounded(f2 v) {
  const float2 w = halves(v), y = make_float2(rsqrtf(w.x), rsqrtf(w.y));
  const f2 y2 = pair(y.x, y.y), n2 = pair(-y.x, -y.y), s = mul2(v, y2);
  const float2 r = halves(fma2(mul2(y2, splat(0.5f)), fma2(fma2(v, n2, s), y2, fma2(s, n2, splat(1.0f))), y2));
  return pair(r.x == r.x ? r.x : y.x, r.y == r.y ? r.y : y.y);
}

// ------------------------------------------------------------------------------------------------
// All kernels of the layers are launched programmatically: a kernel's blocks may be brought up when every block of
// the one before has called launch_next() or ended, beside its last blocks, and wait_previous() holds them until it is
// complete and what it wrote is visible.  Every kernel begins with in_turn(), before it reads or writes memory (the
// column sums behind a product do so at their end), so that a kernel is complete only when all before it are, and no
// kernel comes up before the last but one is complete.  Behind any other kernel this is an ordinary launch.
// (Calls back to back: linear on 16 rows, 1024 to 4096, 5.0 us for 6.15; layer norm and restore of 16384 x 1024 24.9 for
// 29.3.)
__device__ __forceinline__ void launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void in_turn() {
  wait_previous();
  launch_next();
}

// Sums of `parts` partial rows of `width` fp32 columns, in a fixed order; columns below `split` go to lo,
// the others to hi.  A block of 1024 threads has COLS columns, 16 (two sectors of a row, and twice the threads to
// a column) where 32 would leave SMs without a block.
template <typename G, int COLS>
static __global__ void __launch_bounds__(1024) k_sum_parts(const float* __restrict__ part, int64_t parts, int64_t width, int64_t split,
                                                           G* __restrict__ lo, G* __restrict__ hi) {
  constexpr int kRows = 1024 / COLS;
  __shared__ float red[kRows][COLS + 1];
  const int col = threadIdx.x % COLS, row = threadIdx.x / COLS;
  const int64_t c = (int64_t)blockIdx.x * COLS + col;
  in_turn();
  float s = 0.0f;
  if (c < width) {
#pragma unroll 8
    for (int64_t p = row; p < parts; p += kRows) s += part[p * width + c];
  }
  red[row][col] = s;
  __syncthreads();
  const int lane = threadIdx.x & 31, mine = threadIdx.x >> 5;  // a warp's column
  if (mine >= COLS) return;
  const float t = warp_sum(COLS == 32 ? red[lane][mine] : red[lane][mine] + red[lane + kRows / 2][mine]);
  const int64_t o = (int64_t)blockIdx.x * COLS + mine;
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
// What a kernel that gave up waiting leaves, in the current device's status word (NULL: a CUDA error).
constexpr unsigned kStatusGaveUp = 1u;
unsigned int* status_word();
uint32_t stall_bytes();  // the test hook's

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
  auto go = [&](auto cols) {
    constexpr int kCols = decltype(cols)::value;
    return launch_after(k_sum_parts<G, kCols>, dim3((unsigned)ceil_div(width, kCols)), 1024, s, part, parts, width, split, static_cast<G*>(lo),
                        static_cast<G*>(hi));
  };
  return ceil_div(width, 32) < sm_count() ? go(std::integral_constant<int, 16>{}) : go(std::integral_constant<int, 32>{});
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
