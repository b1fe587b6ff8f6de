// unaligned.cuh -- rows of any alignment in groups of eight columns: aligned 16-byte vectors, shifted.
#pragma once

#include "dropout.cuh"

namespace onebit {
namespace layers {

__device__ __forceinline__ uint32_t lanes_of(int width) {  // the lanes of this lane's group of `width`
  return width == 32 ? 0xffffffffu : ((1u << width) - 1) << (threadIdx.x & 31 & ~(width - 1));
}

// A group's words from the aligned vectors that it touches (one more than it fills), m bytes of which lie before it.
template <typename T>
__device__ __forceinline__ void shift_words(uint32_t (&w)[2 * sizeof(T) + 4], int m) {
  constexpr int n = 2 * (int)sizeof(T);
#pragma unroll
  for (int i = 0; i < n + 2; ++i) w[i] = m & 8 ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < n + 1; ++i) w[i] = m & 4 ? w[i + 1] : w[i];
  if (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < n; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], (m & 2) * 8);
  }
}
// Eight columns from c on of a row, 0 past its end.  A vector that reaches over either end of the row
// is read by single elements.
template <typename T, bool VEC>
__device__ __forceinline__ void load_columns(const T* row, int c, int cols, f2 (&f)[4]) {
  if (VEC) {
    if (c < cols) expand8(load8(row + c), f);
    return;
  }
  constexpr int kSize = (int)sizeof(T), n = 2 * kSize;
  uint32_t w[n + 4];
#pragma unroll
  for (int i = 0; i < n + 4; ++i) w[i] = 0;
  const int m = (int)(reinterpret_cast<uintptr_t>(row) & 15), left = m + (cols - c) * kSize;
  const char* const from = reinterpret_cast<const char*>(row + c) - m;
#pragma unroll
  for (int v = 0; v < n / 4 + 1; ++v) {
    if (c >= cols || left <= 16 * v || (v == n / 4 && m == 0)) continue;
    if (left >= 16 * v + 16 && (v > 0 || c > 0 || m == 0)) {
      const uint4 t = __ldg(reinterpret_cast<const uint4*>(from) + v);
      w[4 * v] = t.x, w[4 * v + 1] = t.y, w[4 * v + 2] = t.z, w[4 * v + 3] = t.w;
    } else {
#pragma unroll
      for (int e = 0; e < 16; e += kSize) {
        if (16 * v + e >= left || (v == 0 && c == 0 && e < m)) continue;
        if (kSize == 2) w[4 * v + e / 4] |= (uint32_t)__ldg(reinterpret_cast<const uint16_t*>(from + 16 * v + e)) << (e % 4 * 8);
        else w[4 * v + e / 4] = __ldg(reinterpret_cast<const uint32_t*>(from + 16 * v + e));
      }
    }
  }
  shift_words<T>(w, m);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kSize == 2) f[i] = widen<T>(w[i]);
    else f[i] = pair(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
  }
}
// Eight columns from c on of a row of an output.  All lanes of a row's group come here together.
template <typename T, int TPR, bool VEC>
__device__ __forceinline__ void store_columns(T* row, int c, int cols, const f2 (&f)[4]) {
  if (VEC) {
    if (c < cols) store8(row + c, f);
    return;
  }
  constexpr int kSize = (int)sizeof(T), n = kSize * 2, kWidth = TPR < 32 ? TPR : 32;  // n: words
  uint32_t w[n + 4];  // the last four words of the lane before, then this lane's
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kSize == 2) {
      w[4 + i] = narrow<T>(f[i]);
    } else {
      const float2 h = halves(f[i]);
      w[4 + 2 * i] = __float_as_uint(h.x), w[5 + 2 * i] = __float_as_uint(h.y);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = __shfl_up_sync(lanes_of(kWidth), w[n + i], 1, kWidth);
  if (c >= cols) return;
  const int lane = threadIdx.x & (kWidth - 1), m = (int)(reinterpret_cast<uintptr_t>(row) & 15), left = cols - c;
  // vector v has this lane's elements before (16 v + 16 - m) / kSize; the last m / kSize go with the next lane's
  bool whole[n / 4];
  uint32_t x[n + 4];
#pragma unroll
  for (int i = 0; i < n + 4; ++i) x[i] = w[i];
  const int sh = 16 - m;
#pragma unroll
  for (int i = 0; i < n; ++i) x[i] = sh & 16 ? x[i + 4] : x[i];
  if (!(sh & 16)) {
#pragma unroll
    for (int i = 0; i < n + 2; ++i) x[i] = sh & 8 ? x[i + 2] : x[i];
#pragma unroll
    for (int i = 0; i < n + 1; ++i) x[i] = sh & 4 ? x[i + 1] : x[i];
    if (kSize == 2) {
#pragma unroll
      for (int i = 0; i < n; ++i) x[i] = __funnelshift_r(x[i], x[i + 1], (sh & 2) * 8);
    }
  }
  char* const to = reinterpret_cast<char*>(row + c) - m;
#pragma unroll
  for (int v = 0; v < n / 4; ++v) {
    whole[v] = left * kSize >= 16 * v + 16 - m && (v > 0 || lane > 0 || m == 0);
    if (whole[v]) *reinterpret_cast<uint4*>(to + 16 * v) = make_uint4(x[4 * v], x[4 * v + 1], x[4 * v + 2], x[4 * v + 3]);
  }
  const bool last = lane == kWidth - 1 || c + 8 >= cols;  // no lane behind takes this one's last elements
  if ((last && m > 0) || !whole[0] || !whole[n / 4 - 1]) {
    auto put = [&](int at, uint32_t word, int e) {  // element e of a word's two or one
      if constexpr (kSize == 2) reinterpret_cast<uint16_t*>(row)[at] = (uint16_t)(e ? word >> 16 : word);
      else reinterpret_cast<uint32_t*>(row)[at] = word;
    };
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int v = (e * kSize + m) / 16;
      const bool vector = v < n / 4 ? (v == 0 ? whole[0] : whole[n / 4 - 1]) : !last;
      if (e < left && !vector) put(c + e, w[4 + e * kSize / 4], kSize == 2 ? e & 1 : 0);
    }
    if (!whole[0] && lane > 0) {  // the row ends inside the vector that the lane before counts on
#pragma unroll
      for (int e = 8 - 16 / kSize < 0 ? 0 : 8 - 16 / kSize; e < 8; ++e)
        if ((8 - e) * kSize <= m) put(c + e - 8, w[4 + e * kSize / 4 - n], kSize == 2 ? e & 1 : 0);
    }
  }
}

}  // namespace layers
}  // namespace onebit
