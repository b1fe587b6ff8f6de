// dropout.cuh -- which elements dropout keeps: a counter-based generator, so that any kernel can draw an element's bits
// again from its place in the matrix.
#pragma once

#include <math.h>

#include "layers_common.cuh"

namespace onebit {
namespace layers {

// Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011): ten rounds of two
// 32 x 32 bit products whose halves are exchanged and mixed with the round's key.
__device__ __forceinline__ uint4 philox(uint4 c, uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = (uint64_t)0xD2511F53u * c.x, b = (uint64_t)0xCD9E8D57u * c.z;
    c = make_uint4((uint32_t)(b >> 32) ^ c.y ^ k0, (uint32_t)b, (uint32_t)(a >> 32) ^ c.w ^ k1, (uint32_t)a);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return c;
}

// A call's dropout, as the host passes it.
struct Dropout {
  const int64_t* key;
  uint32_t site;
  uint32_t threshold;  // 0: nothing is dropped, and the key is not read
  float factor;
};
// With the key read, in a kernel.
struct Generator {
  uint32_t k0, k1, step, site, threshold;
  float factor;
  __device__ __forceinline__ explicit Generator(const Dropout& d) : k0(0), k1(0), step(0), site(d.site), threshold(d.threshold), factor(d.factor) {
    if (threshold) {
      const uint64_t seed = (uint64_t)d.key[0];
      k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32), step = (uint32_t)(uint64_t)d.key[1];
    }
  }
  // the bits of a group of eight columns
  __device__ __forceinline__ uint4 draw(int64_t group) const {
    return philox(make_uint4((uint32_t)(uint64_t)group, (uint32_t)((uint64_t)group >> 32), step, site), k0, k1);
  }
  // a group's values, 0 where they are dropped (the upper half of a word is compared in place: what lies below it decides nothing)
  __device__ __forceinline__ void keep8(const uint4& w, f2 (&v)[4]) const {
    const uint32_t words[4] = {w.x, w.y, w.z, w.w}, least = threshold << 16;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 h = halves(v[i]);
      v[i] = pair((words[i] << 16) >= least ? h.x : 0.0f, words[i] >= least ? h.y : 0.0f);
    }
  }
  __device__ __forceinline__ void apply8(int64_t group, f2 (&v)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = mul2(v[i], splat(factor));
    keep8(draw(group), v);
  }
};

// The call's dropout, or what is wrong with it.
inline onebit_status_t make_dropout(Dropout* d, float p, const int64_t* key, uint32_t site) {
  const double t = nearbyint(65536.0 * (double)p);
  if (!(p >= 0.0f && t < 65536.0)) return fail(ONEBIT_ERR_INVALID_ARG, "p is negative, NaN or rounds to 1");
  if (t > 0 && !key) return fail(ONEBIT_ERR_INVALID_ARG, "dropout needs a key");
  if (!aligned(key, 8)) return fail(ONEBIT_ERR_INVALID_ARG, "a buffer is not aligned to its type");
  *d = Dropout{key, site, (uint32_t)t, (float)(65536.0 / (65536.0 - t))};
  return ONEBIT_OK;
}

// Eight columns of a row: at once where rows lie on 16 bytes and are whole groups, else one by one (0 past the end).
template <typename T, bool VEC>
__device__ __forceinline__ void load_group(const T* p, int left, f2 (&f)[4]) {
  if (VEC) {
    expand8(load8(p), f);
  } else {
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < left ? to_f(p[e]) : 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = pair(v[2 * e], v[2 * e + 1]);
  }
}
template <typename T, bool VEC>
__device__ __forceinline__ void store_group8(T* p, int left, const f2 (&f)[4]) {
  if (VEC) {
    store8(p, f);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 h = halves(f[e]);
      if (2 * e < left) p[2 * e] = from_f<T>(h.x);
      if (2 * e + 1 < left) p[2 * e + 1] = from_f<T>(h.y);
    }
  }
}

}  // namespace layers
}  // namespace onebit
