// few_rows.cuh -- y = act(x w^T + bias) + residual for up to 32 rows, as generation meets it.
//
// The weight is read once and nothing else counts: bound by its bytes (8.4 MB at 1024 -> 4096: 1.2 us from HBM)
// and by the latency of a launch.  A tile of the products' kernel would be 128 rows of which 16 are there, and
// 32 blocks would pull the weight; here every warp of the GPU pulls a part of it at once.  A block has 8*G
// columns; its eight warps share them G ways and the contraction 8/G ways, and add up in shared memory, in
// order.  Each lane keeps kAhead 16-byte pieces of the weight in flight.  16 x 1024 x 4096: the kernel takes 4.3 us with the
// weight in HBM, 3.4 with it in L2; with gelu, called from Python back to back, 4.9 us, 10.3 by the products' kernel.
//
// The products are 16x8x16 warp instructions.  The contraction index is dealt to them in an order of its own:
// lane (n, q) of a column group holds eight neighbouring k of column n, which are the four pairs that it owes to two
// instructions, so that weights and rows both come as 16-byte loads straight from memory.
#pragma once

#include "linear_common.cuh"

namespace onebit {
namespace layers {

constexpr int kFewRows = 32;
constexpr int kFewThreads = 256;

template <typename T>
__device__ __forceinline__ void mma_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if (sizeof(T) == 2 && std::is_same<T, __half>::value)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

struct FewRowsArgs {
  const void* x;
  int64_t ldx;
  const void* w;
  int64_t ldw;
  const float* bias;
  const void* residual;
  int64_t ldr;
  void* y;
  int64_t ldy;
  int rows, in, out, act;
};

// M: sixteen-row halves (1 or 2); G: column groups of eight in a block.
template <typename T, int M, int G>
__global__ void __launch_bounds__(kFewThreads) k_few_rows(const FewRowsArgs A) {
  in_turn();
  constexpr int kSplits = 8 / G, kAhead = 4;
  __shared__ float part[kSplits][M * 16][G * 8 + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = warp % G, split = warp / G;
  const int n = lane >> 2, q = lane & 3;
  const int col = blockIdx.x * (8 * G) + group * 8 + n;
  // this warp's part of the contraction: whole steps of 32
  const int steps = (A.in + 31) / 32, per = (steps + kSplits - 1) / kSplits;
  const int s0 = split * per, s1 = s0 + per < steps ? s0 + per : steps;
  const T* w = static_cast<const T*>(A.w) + (int64_t)(col < A.out ? col : 0) * A.ldw;
  const T* x = static_cast<const T*>(A.x);
  float d[M][4] = {};
  const uint4 zero = make_uint4(0, 0, 0, 0);
  auto piece = [&](int s) {
    const int k = s * 32 + q * 8;
    return col < A.out && s < s1 && k < A.in ? __ldg(reinterpret_cast<const uint4*>(w + k)) : zero;
  };
  uint4 ahead[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) ahead[i] = piece(s0 + i);
  for (int s = s0; s < s1; s += kAhead) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const uint4 b = ahead[i];
      ahead[i] = piece(s + kAhead + i);
      const int k = (s + i) * 32 + q * 8;
#pragma unroll
      for (int m = 0; m < M; ++m) {
        const int r0 = m * 16 + n, r1 = r0 + 8;
        const bool in = s + i < s1 && k < A.in;
        const uint4 a = in && r0 < A.rows ? __ldg(reinterpret_cast<const uint4*>(x + r0 * A.ldx + k)) : zero;
        const uint4 c = in && r1 < A.rows ? __ldg(reinterpret_cast<const uint4*>(x + r1 * A.ldx + k)) : zero;
        mma_16x8x16<T>(d[m], a.x, c.x, a.y, c.y, b.x, b.y);
        mma_16x8x16<T>(d[m], a.z, c.z, a.w, c.w, b.z, b.w);
      }
    }
  }
  // lane (n, q) has rows n and n + 8, columns 2q and 2q + 1 of its group
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) part[split][m * 16 + n + 8 * (i / 2)][group * 8 + 2 * q + (i & 1)] = d[m][i];
  __syncthreads();
  for (int i = threadIdx.x; i < M * 16 * G * 8; i += kFewThreads) {
    const int r = i / (G * 8), j = i % (G * 8), c = blockIdx.x * (8 * G) + j;
    if (r >= A.rows || c >= A.out) continue;
    float z = part[0][r][j];
#pragma unroll
    for (int s = 1; s < kSplits; ++s) z += part[s][r][j];
    if (A.bias) z += __ldg(A.bias + c);
    float v = act_value(A.act, z);
    if (A.residual) v += to_f(static_cast<const T*>(A.residual)[r * A.ldr + c]);
    static_cast<T*>(A.y)[r * A.ldy + c] = from_f<T>(v);
  }
}

// Few rows, on 16 bytes, and no checkpoint (whose 64-column blocks would span these blocks).
inline bool few_rows(const onebit_linear_t& a) {
  return a.rows <= kFewRows && !a.codes && a.in % 8 == 0 && vec16(a.x, a.ldx) && vec16(a.w, a.ldw);
}
// Groups a block: the fewest with which a warp's part of the contraction fills most of its kAhead pieces in flight, as
// more warps a column shorten its chain; a short contraction leaves them room for more columns, which read x less often.
// us by 1, 2, 4, 8 groups, one row, weights from HBM: 4096 -> 4096 9.0 14.9 23.0 28.8, 1024 -> 4096 3.8 4.7 6.6 8.4,
// 768 -> 4096 3.5 4.3 5.2 6.6, 512 -> 4096 2.9 2.8 3.8 4.8, 256 -> 4096 2.6 2.1 2.1 2.2, 256 -> 8192 4.2 3.3 2.6 2.9,
// 512 -> 1024 1.9 2.1 2.9 3.2.  Very many columns and a small x end that: eight groups (16 rows of 1024 -> 32768 19.3 and
// 16.9, of 1024 -> 20480 13.2 and 15.7; 32 rows of 1024 -> 32768 30.3 and 43.3).
template <typename T>
cudaError_t run_few_rows(const onebit_linear_t& a, cudaStream_t s) {
  const FewRowsArgs f{a.x, a.ldx, a.w, a.ldw, a.bias, a.residual, a.ldr, a.y, a.ldy, (int)a.rows, (int)a.in, (int)a.out, a.activation};
  const int64_t groups = ceil_div(a.out, 8), sms = sm_count();
  auto go = [&](auto m, auto g) {
    constexpr int kM = decltype(m)::value, kG = decltype(g)::value;
    return launch_after(k_few_rows<T, kM, kG>, (unsigned)ceil_div(groups, kG), kFewThreads, s, f);
  };
  using std::integral_constant;
  auto by_rows = [&](auto g) {
    return a.rows <= 16 ? go(integral_constant<int, 1>{}, g) : go(integral_constant<int, 2>{}, g);
  };
  if (groups >= 24 * sms && a.rows <= 16) return by_rows(integral_constant<int, 8>{});
  if (a.in < 384 && groups >= 2 * sms) return by_rows(integral_constant<int, 4>{});
  if (a.in < 640 && groups >= sms) return by_rows(integral_constant<int, 2>{});
  return by_rows(integral_constant<int, 1>{});
}

}  // namespace layers
}  // namespace onebit
