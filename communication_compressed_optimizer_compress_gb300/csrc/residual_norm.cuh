// residual_norm.cuh -- kernels of the residual sum with the norms around it, forward and backward with the parameters'
// gradients.  See include/onebit_layers.h for the formulas.
#pragma once

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "unaligned.cuh"

namespace onebit {
namespace layers {

struct ResidualForward {
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
  unsigned int* status;
  uint32_t stall_tx;  // (clusters) test hook: bytes that every sum waits for and no block sends (normally 0)
};

struct ResidualBackward {
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
  unsigned int* status;
  uint32_t stall_tx;
  float* sums;  // (rows read again:) each row's two sums behind the norm before the next block
};

// ------------------------------------------------------------------------------------------------
// Rows held in registers between their statistics and their outputs, so that they are read once: TPR threads have a row, a
// thread CH groups of eight neighbouring columns (and the same columns of every row that it meets, so that parameters stay
// in registers and their gradients add up there).  What the next rows need is copied ahead into shared memory, each
// thread's own columns into slots of its own, which takes no registers and no barrier (backward reads four rows for each one:
// ahead in registers it would have 16 warps an SM and one row in flight).
//
// Rows that lie on 16 bytes and are whole groups (VEC) are copied and stored as they lie.  Of others a thread copies the aligned
// vectors that its columns touch, one more than they fill, and shifts; their outputs are put together from its own and its
// neighbour's values into aligned vectors, single elements where a warp's columns or the row begin and end.

// One input's rows on their way: IN rows share a stage of the ring, this input has the `in`-th (of two rows at a time: and the one behind it).
template <typename T, int TPR, int CH, bool VEC, int IN, int STAGES, int THREADS, int ROWS = 1>
struct RowStream {
  static constexpr int kOwn = (int)sizeof(T) / 2, kVectors = kOwn + (VEC ? 0 : 1);  // 16-byte vectors of a group
  static constexpr int kBytes = STAGES * IN * CH * kVectors * THREADS * 16;
  const T* base;  // the matrix
  const T* next;  // the row to copy next
  int64_t hop;
  uint32_t slot;
  __device__ __forceinline__ RowStream(char* smem, int in, const void* p, int64_t ld, int64_t first, int64_t step, int t, int cols)
      : base(static_cast<const T*>(p)), next(base + first * ld), hop(step * ld),
        slot((uint32_t)__cvta_generic_to_shared(smem) + ((uint32_t)in * CH * kVectors * THREADS + threadIdx.x) * 16) {
#pragma unroll
    for (int j = 0; j < CH; ++j)
      if ((j * TPR + t) * 8 >= cols) {  // nothing is ever copied there: zeros
#pragma unroll
        for (int i = 0; i < STAGES; ++i)
#pragma unroll
          for (int v = 0; v < kVectors; ++v)
#pragma unroll
            for (int n = 0; n < ROWS; ++n) asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at(i, j, v, n)), "r"(0) : "memory");
      }
  }
  __device__ __forceinline__ uint32_t at(int stage, int j, int v, int n = 0) const {
    return slot + (uint32_t)(stage * (IN * CH * kVectors * THREADS) + ((n * CH + j) * kVectors + v) * THREADS) * 16;
  }
  // the n-th row, n rows (`offset` elements) behind the next one
  __device__ __forceinline__ void ahead(int stage, int t, int cols, int n = 0, int64_t offset = 0) {
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int c = (j * TPR + t) * 8;
      if (c >= cols) continue;
      if (VEC) {
#pragma unroll
        for (int v = 0; v < kVectors; ++v)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at(stage, j, v, n)), "l"(next + offset + c + v * (16 / (int)sizeof(T))) : "memory");
      } else {
        const char* const row = reinterpret_cast<const char*>(next);
        const int m = (int)(reinterpret_cast<uintptr_t>(row) & 15);
        const int left = m + (cols - c) * (int)sizeof(T);  // from the first vector to the row's end
#pragma unroll
        for (int v = 0; v < kVectors; ++v) {
          const int bytes = left - 16 * v < 16 ? left - 16 * v : 16;  // the rest is zeros
          if (v == 0 && c == 0 && row - m < reinterpret_cast<const char*>(base)) {  // what lies before the matrix is left alone
#pragma unroll 1
            for (int e = 0; e < 16; e += (int)sizeof(T)) {
              uint32_t bits = 0;
              if (e >= m && e < bytes) {
                if (sizeof(T) == 2) bits = *reinterpret_cast<const uint16_t*>(row - m + e);
                else bits = *reinterpret_cast<const uint32_t*>(row - m + e);
              }
              if (sizeof(T) == 2) asm volatile("st.shared.b16 [%0], %1;" ::"r"(at(stage, j, v) + e), "h"((uint16_t)bits) : "memory");
              else asm volatile("st.shared.b32 [%0], %1;" ::"r"(at(stage, j, v) + e), "r"(bits) : "memory");
            }
          } else {
            const bool some = bytes > 0;
            asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(at(stage, j, v)), "l"(some ? row - m + (int64_t)c * (int)sizeof(T) + 16 * v : row - m),
                         "r"(some ? bytes : 0)
                         : "memory");
          }
        }
      }
    }
    if (ROWS == 1) next += hop;
  }
  // eight columns of a row, 0 past the end; m: the row's distance from 16 bytes (VEC: any)
  __device__ __forceinline__ void take(int stage, int j, int m, f2 (&f)[4], int n = 0) const {
    uint32_t w[4 * kVectors];
#pragma unroll
    for (int v = 0; v < kVectors; ++v)
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[4 * v]), "=r"(w[4 * v + 1]), "=r"(w[4 * v + 2]), "=r"(w[4 * v + 3]) : "r"(at(stage, j, v, n)) : "memory");
    if constexpr (!VEC) shift_words<T>(w, m);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 2) f[i] = widen<T>(w[i]);
      else f[i] = pair(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    }
  }
};
template <typename T>
__device__ __forceinline__ int off16(const void* p, int64_t ld, int64_t r) {  // a row's distance from 16 bytes
  return (int)((uint32_t)reinterpret_cast<uintptr_t>(p) + (uint32_t)r * (uint32_t)ld * (uint32_t)sizeof(T)) & 15;
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// a parameter's eight columns, `none` where there is no parameter, 0 past the end
__device__ __forceinline__ void held8(const float* p, int c, int cols, float none, f2 (&f)[4]) {
  if (!p) {
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = pair(c + 2 * e < cols ? none : 0.0f, c + 2 * e + 1 < cols ? none : 0.0f);
  } else if ((reinterpret_cast<uintptr_t>(p) & 15) == 0 && c + 8 <= cols) {
    expand8(load8(p + c), f);
  } else {
    load_group<float, false>(p + c, cols - c, f);
  }
}

// Sums over the TPR threads of a row, the same order on every call; every thread gets them.  `red` has room for two sets,
// used alternately, so that one barrier a call is enough.
template <int TPR, int N>
constexpr int kRedWords = TPR > 32 ? N * TPR / 32 : 4;
template <int TPR, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*red)[kRedWords<TPR, N>], int& turn, int bar) {
  constexpr int kWidth = TPR < 32 ? TPR : 32;
  if constexpr (N == 2 && TPR > 32) {  // each half of the warp goes on with one of the two: five exchanges for ten
    const bool upper = threadIdx.x & 16;
    float u = (upper ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, upper ? v[0] : v[1], 16);
#pragma unroll
    for (int o = 8; o; o >>= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
    v[0] = u;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int o = kWidth / 2; o; o >>= 1) v[i] += __shfl_xor_sync(lanes_of(kWidth), v[i], o);
  }
  if constexpr (TPR > 32) {
    constexpr int kWarps = TPR / 32;
    float* r = red[turn];
    turn ^= 1;
    if ((threadIdx.x & (32 / N - 1)) == 0) r[(threadIdx.x & 31) / (32 / N) * kWarps + (threadIdx.x % TPR >> 5)] = v[0];
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "n"(TPR) : "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (kWarps % 4 == 0) {
        v[i] = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; w += 4) {
          const float4 q = *reinterpret_cast<const float4*>(r + i * kWarps + w);
          v[i] += (q.x + q.y) + (q.z + q.w);
        }
      } else {
        const float2 q = *reinterpret_cast<const float2*>(r + i * kWarps);
        v[i] = q.x + q.y;
      }
    }
  }
}

// Rows of more columns than a block holds are a cluster's: each block has a part of the columns.
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_blocks() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_barrier() { asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory"); }
constexpr int kClusterMost = 8;

// The blocks' sums of a row to its sum, added in the blocks' order: each block sends its own to all, who wait for the bytes.  (With
// the cluster's barrier instead, whose release waits for the rows that were stored before it, a row of 8192 columns took 2 us a sum.)
// Two sets of places take turns: a block sends to one of them again only after it has had what the others sent behind their reading it.
//
// A wait ends after about a second, or as soon as another thread of the block has given up the same one; the status word says so.  The
// phase that was waited for stays open, so its barrier is not touched again: behind the barrier of the block's next sums every thread sees
// which wait was given up, and from there on none arrives, sends or waits: what is left of the rows is done on sums that say nothing.
// The other blocks of the cluster then miss what this one would have sent, and their next wait ends the same way.  (Each of the three
// has the condition to itself: behind one branch around them, or with the rows left, backward's loads for the next row no longer overlap
// the sums, and 4096 x 8192 with RMS norms on both sides takes 160 us for 111.)
template <int N>
struct ClusterSums {
  struct Shared {
    float from[2][kClusterMost][N];
    uint64_t bar[2];
    uint32_t gave_up;  // 0, or the number of the wait that ran out, from 1 on
  };
  Shared& m;
  unsigned int* status;
  uint32_t stall, rank, blocks, count;
  bool mine;  // this thread's wait ran out
  // by all threads, before the cluster's first barrier
  __device__ __forceinline__ ClusterSums(Shared& shared, unsigned int* status_, uint32_t stall_)
      : m(shared), status(status_), stall(stall_), rank(cluster_rank()), blocks(cluster_blocks()), count(0), mine(false) {
    if (threadIdx.x == 0) {
      for (int i = 0; i < 2; ++i) asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(at(&m.bar[i])) : "memory");
      *(volatile uint32_t*)&m.gave_up = 0;
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncwarp();
  }
  __device__ __forceinline__ static uint32_t at(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
  __device__ __forceinline__ bool here(uint32_t bar, uint32_t parity) const {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
  }
  // Behind the block's own sums, whose barrier all threads have just passed: all see the same wait before this one given up, or none.
  // `turn` is the set of places, alternating from 0.
  __device__ __forceinline__ void operator()(float (&v)[N], int turn) {
    const uint32_t parity = count >> 1 & 1, bar = at(&m.bar[turn]);
    ++count;
    const uint32_t lost = *(volatile uint32_t*)&m.gave_up;
    const bool live = lost == 0 || lost == count;  // (another thread may be giving up this very wait already)
    if (live && threadIdx.x == 0) asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(blocks * N * 4 + stall) : "memory");
    if (live && threadIdx.x < blocks) {
      uint32_t to, its;
      asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(at(&m.from[turn][rank][0])), "r"(threadIdx.x));
      asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(its) : "r"(bar), "r"(threadIdx.x));
#pragma unroll
      for (int i = 0; i < N; ++i)
        asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(to + 4 * i), "r"(__float_as_uint(v[i])), "r"(its) : "memory");
    }
    __syncwarp();
    if (live && !here(bar, parity)) {
      const long long t0 = clock64();
      while (!here(bar, parity)) {
        if (*(volatile uint32_t*)&m.gave_up) {
          mine = true;
          break;
        }
        if (clock64() - t0 > 2000000000ll) {
          *(volatile uint32_t*)&m.gave_up = count;
          atomicOr(status, kStatusGaveUp);
          mine = true;
          break;
        }
      }
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = *(volatile float*)&m.from[turn][0][i];
      for (uint32_t b = 1; b < blocks; ++b) v[i] += *(volatile float*)&m.from[turn][b][i];
    }
  }
  // No block leaves while another may still send to it.  One that has had all that it waited for has nothing more coming; one
  // that gave up stays for some ten milliseconds more behind all the cluster's last sends.
  __device__ __forceinline__ void end() const {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
    if (mine) {
      const long long t0 = clock64();
      while (clock64() - t0 < 20000000ll) {
      }
    }
  }
};

struct OneBlock {
  template <class Shared>
  __device__ __forceinline__ OneBlock(Shared&, unsigned int*, uint32_t) {}
  template <int N>
  __device__ __forceinline__ void operator()(float (&)[N], int) const {}
  __device__ __forceinline__ void end() const {}
};

// v becomes its distance from the mean, columns past the end stay 0; returns its squares' sum
template <int TPR, int CH, bool VEC>
__device__ __forceinline__ float centre(f2 (&v)[CH][4], float mean, int t, int cols) {
  f2 s = 0;
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    const int c = (j * TPR + t) * 8;
    const f2 shift = splat(c < cols ? -mean : 0.0f);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[j][e] = add2(v[j][e], VEC ? shift : pair(c + 2 * e < cols ? -mean : 0.0f, c + 2 * e + 1 < cols ? -mean : 0.0f));
      s = fma2(v[j][e], v[j][e], s);
    }
  }
  return sum_of(s);
}
template <int CH>
__device__ __forceinline__ float squares(const f2 (&v)[CH][4]) {
  f2 s = 0;
#pragma unroll
  for (int j = 0; j < CH; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) s = fma2(v[j][e], v[j][e], s);
  return sum_of(s);
}
template <int CH>
__device__ __forceinline__ float total(const f2 (&v)[CH][4]) {
  f2 s = 0;
#pragma unroll
  for (int j = 0; j < CH; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) s = add2(s, v[j][e]);
  return sum_of(s);
}

template <int TPR>
constexpr int kForwardThreads = TPR > 128 ? TPR : 128;
// Blocks that an SM has room for at least: 72 registers a thread where one group of columns of one row is held, 80 with a norm behind the block, 96 for two rows (a
// norm behind the block: 128), else 128.
template <int TPR, int CH, int NR, bool POST>
constexpr int kForwardBlocks = (CH > 1 ? 512 : NR > 1 ? (POST ? 512 : 640) : POST ? 768 : 896) / kForwardThreads<TPR>;
template <typename T>
constexpr int kForwardStages = sizeof(T) == 2 ? 3 : 2;

// One pass over the rows: the block's statistics (where a norm stands behind it), its masked and gated values onto x, s's statistics, y.
// Variances are summed about the mean, a second exchange behind the first.  NR rows at a time: two share the exchanges of their sums,
// the barrier behind them and the reciprocal roots.  16384 x 1024 bf16, over twelve placements in memory: layer norm 23.1 us and RMS norm
// 22.4, 134 MB at 5.8 and 6.0 TB/s; with dropout 25.9 and 23.3, with RMS norms on both sides, gate and dropout 26.2.  Then bound by
// latency, with the 16 to 24 warps an SM that registers leave: 56 to 61% of the issue slots, no pipe above 45%.  Odd rows (1001: 61.5) are bound by
// their shifts' instructions, 2.7 times as many: 68% of the issue slots, the ALU 59%.  fp32 (layer norms, gate, dropout: 62, floor 40) by latency
// too (issue 40%): a copy of 16 of a thread's 32 bytes asks for half a sector, so that the L2 has three times the requests for twice the bytes.
template <typename T, int TPR, int CH, int NR, bool VEC, bool POST, bool CLUSTER>
static __global__ void __launch_bounds__(kForwardThreads<TPR>, kForwardBlocks<TPR, CH, NR, POST>) k_rn_forward(const ResidualForward A) {
  static_assert(NR == 1 || (VEC && !CLUSTER), "two rows at a time: dense ones of one block");
  constexpr int kThreads = kForwardThreads<TPR>, kGroups = kThreads / TPR, kStages = kForwardStages<T>;
  extern __shared__ __align__(16) char dynamic[];
  __shared__ __align__(16) float red[kGroups][2][kRedWords<TPR, NR>];
  __shared__ typename ClusterSums<NR>::Shared places;
  const uint32_t rank = CLUSTER ? cluster_rank() : 0, blocks = CLUSTER ? cluster_blocks() : 1;
  const int t = threadIdx.x % TPR + rank * TPR * CH, group = threadIdx.x / TPR, cols = A.cols;
  const int64_t step = (int64_t)(gridDim.x / blocks) * kGroups * NR, first = ((int64_t)(blockIdx.x / blocks) * kGroups + group) * NR;
  using Stream = RowStream<T, TPR, CH, VEC, 2 * NR, kStages, kThreads, NR>;
  Stream x(dynamic, 0, A.x, A.ldx, first, step, t, cols), b(dynamic, NR, A.block, A.ldblock, first, step, t, cols);
  const bool block = A.block != nullptr;
  std::conditional_t<CLUSTER, ClusterSums<NR>, OneBlock> across(places, A.status, A.stall_tx);
  if (CLUSTER) cluster_barrier();  // the other blocks are there to be sent to
  in_turn();
  if (first >= A.rows) return;     // (no barrier is the whole block's, and a cluster's blocks have the same rows)
  auto ahead = [&](int stage, int64_t r) {
    if (r < A.rows) {
#pragma unroll
      for (int n = 0; n < NR; ++n)
        if (n == 0 || r + n < A.rows) {
          x.ahead(stage, t, cols, n, n * A.ldx);
          if (block) b.ahead(stage, t, cols, n, n * A.ldblock);
        }
      if (NR > 1) x.next += x.hop, b.next += b.hop;
    }
    copies_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) ahead(i, first + i * step);
  const Generator gen(A.drop);
  // what the block's values are multiplied by (dropout's factor included) and what is added behind its norm, gamma, beta
  f2 pa[CH][4], pb[CH][4], gamma[CH][4], beta[CH][4];
  const f2 scale = splat(A.scale * (gen.threshold ? gen.factor : 1.0f));
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    const int c = (j * TPR + t) * 8;
    held8(A.gate, c, cols, 1.0f, pa[j]);
#pragma unroll
    for (int e = 0; e < 4; ++e) pa[j][e] = mul2(pa[j][e], scale);
    if (POST) {
      f2 g[4];
      held8(A.block_beta, c, cols, 0.0f, pb[j]);
      held8(A.block_gamma, c, cols, 1.0f, g);
#pragma unroll
      for (int e = 0; e < 4; ++e) pb[j][e] = mul2(pb[j][e], pa[j][e]), pa[j][e] = mul2(pa[j][e], g[e]);
    }
    held8(A.gamma, c, cols, 0.0f, gamma[j]);
    held8(A.beta, c, cols, 0.0f, beta[j]);
  }
  int turn = 0, stage = 0;
  T *ps = static_cast<T*>(A.s) + first * A.lds, *py = static_cast<T*>(A.y) + first * A.ldy;
  // v becomes v - mean; out 1/sqrt of its mean square
  auto normal = [&](f2(&v)[NR][CH][4], float* means, float* rstds, int64_t r, float(&rstd)[NR]) {
    float q[NR];
    auto sums = [&] {
      const int now = turn;
      row_sums<TPR>(q, red[group], turn, 1 + group);
      across(q, now);
    };
    if (A.layer) {
#pragma unroll
      for (int n = 0; n < NR; ++n) q[n] = total(v[n]);
      sums();
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        const float mean = q[n] * A.inv_cols;
        if (t == 0 && (n == 0 || r + n < A.rows)) means[r + n] = mean;
        q[n] = centre<TPR, CH, VEC>(v[n], mean, t, cols);
      }
    } else {
#pragma unroll
      for (int n = 0; n < NR; ++n) q[n] = squares(v[n]);
    }
    sums();
    const float2 root = halves(rsqrt_rounded(fma2(pair(q[0], q[NR - 1]), splat(A.inv_cols), splat(A.eps))));
    rstd[0] = root.x, rstd[NR - 1] = root.y;
#pragma unroll
    for (int n = 0; n < NR; ++n)
      if (t == 0 && (n == 0 || r + n < A.rows)) rstds[r + n] = rstd[n];
  };
  for (int64_t r = first; r < A.rows; r += step) {  // (a second row that is not there has no outputs)
    copies_wait<kStages - 2>();
    ahead(stage == 0 ? kStages - 1 : stage - 1, r + (kStages - 1) * step);
    f2 s[NR][CH][4];
    const int mx = VEC ? 0 : off16<T>(A.x, A.ldx, r), mb = VEC ? 0 : off16<T>(A.block, A.ldblock, r);
    uint4 bits[NR][CH];
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        bits[n][j] = gen.threshold ? gen.draw((r + n) * A.groups + j * TPR + t) : make_uint4(0, 0, 0, 0);
        x.take(stage, j, mx, s[n][j], n);
      }
    if (block) {
      f2 v[NR][CH][4];
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int j = 0; j < CH; ++j) b.take(stage, j, mb, v[n][j], n);
      float rstd[NR];
      if (POST) normal(v, A.block_mean, A.block_rstd, r, rstd);
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int j = 0; j < CH; ++j) {
          const int c = (j * TPR + t) * 8;
#pragma unroll
          for (int e = 0; e < 4; ++e) v[n][j][e] = POST ? fma2(mul2(v[n][j][e], splat(rstd[n])), pa[j][e], pb[j][e]) : mul2(v[n][j][e], pa[j][e]);
          if (gen.threshold) gen.keep8(bits[n][j], v[n][j]);
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][j][e] = add2(s[n][j][e], v[n][j][e]);
          if (n == 0 || r + n < A.rows) store_columns<T, TPR, VEC>(ps + n * A.lds, c, cols, s[n][j]);
        }
      ps += step * A.lds;
    }
    if (A.gamma) {
      float rstd[NR];
      normal(s, A.mean, A.rstd, r, rstd);
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int j = 0; j < CH; ++j) {
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][j][e] = fma2(mul2(s[n][j][e], splat(rstd[n])), gamma[j][e], beta[j][e]);
          if (n == 0 || r + n < A.rows) store_columns<T, TPR, VEC>(py + n * A.ldy, (j * TPR + t) * 8, cols, s[n][j]);
        }
      py += step * A.ldy;
    }
    if (++stage == kStages) stage = 0;
  }
  copies_wait<0>();
  across.end();
}

constexpr int kBackwardThreads = 512;  // of 128 registers: all that an SM has room for, so that it leaves one part
template <typename T, bool VEC>
constexpr int kBackwardStages = sizeof(T) == 2 ? 3 : VEC ? 3 : 2;

// What the block's side has: nothing but dropout and a scale, a gate, or a norm (and a gate).
enum BlockSide { kBlockPlain = 0, kBlockGate = 1, kBlockNorm = 2 };
// RMS: the norms are known to be without means (else A.layer says so), which saves their sums.
// One pass over the rows: what comes through the norm before the next block joins ds to t, which goes on through mask, gate and the norm
// behind the block; a thread adds up its columns' part of the parameters' gradients.  Bound by latency, 16 warps an SM (49 to 59% of the issue
// slots, no pipe above 49%): 16384 x 1024 bf16 36.2 us with layer norm and dropout, parameters' sums included (168 MB at 4.6 TB/s), 32.8 with RMS norm; 8192 x 2048
// f16 with RMS norms on both sides, gate and dropout 46.1 (the means' sums cost 15 more).  640 threads of 96 registers are no faster.  Odd rows
// (1001: 69) by their shifts' instructions, as forward; fp32 (RMS norm 80.5, floor 50; everything 105, floor 60) waits for its copies, issue 15 to
// 29%, with four times the L2 requests of 16 bits for twice the bytes.
template <typename T, int TPR, bool VEC, int SIDE, bool CLUSTER, bool RMS>
static __global__ void __launch_bounds__(kBackwardThreads, 1) k_rn_backward(const ResidualBackward A) {
  constexpr int kGroups = kBackwardThreads / TPR, kStages = kBackwardStages<T, VEC>;
  constexpr bool POST = SIDE == kBlockNorm, block = SIDE != kBlockPlain;
  constexpr int kSums = RMS ? 1 : 2;                                   // of a row behind each norm
  constexpr int kKinds = kSums + (SIDE == kBlockGate ? 1 : SIDE / 2 * kSums);  // over the rows: of dy shat, dy, d bhat, d; without the means' none of dy and d
  extern __shared__ __align__(16) char dynamic[];
  __shared__ __align__(16) float red[kGroups][2][kRedWords<TPR, kSums>];
  __shared__ typename ClusterSums<kSums>::Shared places;
  const uint32_t rank = CLUSTER ? cluster_rank() : 0, blocks = CLUSTER ? cluster_blocks() : 1;
  const int t = threadIdx.x % TPR + rank * TPR, group = threadIdx.x / TPR, cols = A.cols, c = t * 8;
  const int64_t step = (int64_t)(gridDim.x / blocks) * kGroups, first = (int64_t)(blockIdx.x / blocks) * kGroups + group;
  using Stream = RowStream<T, TPR, 1, VEC, 4, kStages, kBackwardThreads>;
  Stream dy(dynamic, 0, A.dy, A.lddy, first, step, t, cols), s(dynamic, 1, A.s, A.lds, first, step, t, cols),
      ds(dynamic, 2, A.ds, A.ldds, first, step, t, cols), b(dynamic, 3, A.block, A.ldblock, first, step, t, cols);
  const bool pre = A.gamma != nullptr, path = A.ds != nullptr;
  std::conditional_t<CLUSTER, ClusterSums<kSums>, OneBlock> across(places, A.status, A.stall_tx);
  if (CLUSTER) cluster_barrier();  // the other blocks are there to be sent to
  in_turn();
  auto ahead = [&](int stage, int64_t r) {
    if (r < A.rows) {
      if (pre) dy.ahead(stage, t, cols), s.ahead(stage, t, cols);
      if (path) ds.ahead(stage, t, cols);
      if (block) b.ahead(stage, t, cols);
    }
    copies_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) ahead(i, first + i * step);
  const Generator gen(A.drop);
  f2 gamma[4], pa[4], sum[kKinds][4];
  held8(A.gamma, c, cols, 0.0f, gamma);
  if (block) held8(A.gate, c, cols, 1.0f, pa);
  if (POST) {
    f2 g[4];
    held8(A.block_gamma, c, cols, 1.0f, g);
#pragma unroll
    for (int e = 0; e < 4; ++e) pa[e] = mul2(pa[e], g[e]);
  }
  const f2 scale = splat(A.scale * (gen.threshold ? gen.factor : 1.0f));
#pragma unroll
  for (int k = 0; k < kKinds; ++k)
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[k][e] = 0;
  const bool layer = !RMS && A.layer;
  float mean = 0.0f, rstd = 0.0f, block_mean = 0.0f, block_rstd = 0.0f;  // of the next row
  auto statistics = [&](int64_t r) {
    if (r >= A.rows) return;
    if (pre) {
      if (layer) mean = __ldg(A.mean + r);
      rstd = __ldg(A.rstd + r);
    }
    if (POST) {
      if (layer) block_mean = __ldg(A.block_mean + r);
      block_rstd = __ldg(A.block_rstd + r);
    }
  };
  statistics(first);
  int turn = 0, stage = 0;
  auto sums = [&](float(&v)[kSums]) {
    const int now = turn;
    row_sums<TPR>(v, red[group], turn, 1 + group);
    across(v, now);
  };
  T *pdx = static_cast<T*>(A.dx) + first * A.lddx, *pdb = static_cast<T*>(A.dblock) + first * A.lddblock;
  for (int64_t r = first; r < A.rows; r += step) {
    const float mu = mean, rs = rstd, bmu = block_mean, brs = block_rstd;
    copies_wait<kStages - 2>();
    ahead(stage == 0 ? kStages - 1 : stage - 1, r + (kStages - 1) * step);
    statistics(r + step);
    const uint4 bits = gen.threshold ? gen.draw(r * A.groups + t) : make_uint4(0, 0, 0, 0);  // (beside the first sums' exchanges)
    f2 d[4];  // t, then d, then what is left of it before the block
    if (path) {
      ds.take(stage, 0, VEC ? 0 : off16<T>(A.ds, A.ldds, r), d);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) d[e] = 0;
    }
    if (pre) {
      f2 q[4], hat[4], s0 = 0, s1 = 0;
      dy.take(stage, 0, VEC ? 0 : off16<T>(A.dy, A.lddy, r), q);
      s.take(stage, 0, VEC ? 0 : off16<T>(A.s, A.lds, r), hat);
#pragma unroll
      for (int e = 0; e < 4; ++e) {  // columns past the end have dy = gamma = 0 and add nothing
        hat[e] = mul2(RMS ? hat[e] : add2(hat[e], splat(-mu)), splat(rs));
        sum[0][e] = fma2(q[e], hat[e], sum[0][e]);
        if (!RMS) sum[kSums - 1][e] = add2(sum[kSums - 1][e], q[e]);
        q[e] = mul2(q[e], gamma[e]);
        if (!RMS) s0 = add2(s0, q[e]);
        s1 = fma2(q[e], hat[e], s1);
      }
      float v[kSums];
      v[0] = sum_of(s0), v[kSums - 1] = sum_of(s1);
      sums(v);
      const f2 m0 = splat(layer ? -v[0] * A.inv_cols * rs : 0.0f), m1 = splat(-v[kSums - 1] * A.inv_cols * rs);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const f2 scaled = RMS ? mul2(q[e], splat(rs)) : fma2(q[e], splat(rs), m0);
        d[e] = add2(fma2(hat[e], m1, scaled), d[e]);
      }
    }
    store_columns<T, TPR, VEC>(pdx, c, cols, d);
    pdx += step * A.lddx;
    if (A.dblock) {
#pragma unroll
      for (int e = 0; e < 4; ++e) d[e] = mul2(d[e], scale);
      if (gen.threshold) gen.keep8(bits, d);
      if (block) {
        f2 hat[4];
        b.take(stage, 0, VEC ? 0 : off16<T>(A.block, A.ldblock, r), hat);
        if (POST) {
          f2 s0 = 0, s1 = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) {  // d is not 0 past the end, where pa is, and its sums there go nowhere
            hat[e] = mul2(RMS ? hat[e] : add2(hat[e], splat(-bmu)), splat(brs));
            sum[kSums][e] = fma2(d[e], hat[e], sum[kSums][e]);
            if (!RMS) sum[kKinds - 1][e] = add2(sum[kKinds - 1][e], d[e]);
            d[e] = mul2(d[e], pa[e]);
            if (!RMS) s0 = add2(s0, d[e]);
            s1 = fma2(d[e], hat[e], s1);
          }
          float v[kSums];
          v[0] = sum_of(s0), v[kSums - 1] = sum_of(s1);
          sums(v);
          const f2 m0 = splat(layer ? -v[0] * A.inv_cols * brs : 0.0f), m1 = splat(-v[kSums - 1] * A.inv_cols * brs);
#pragma unroll
          for (int e = 0; e < 4; ++e) d[e] = fma2(hat[e], m1, RMS ? mul2(d[e], splat(brs)) : fma2(d[e], splat(brs), m0));
        } else {
          if (gen.threshold) gen.keep8(bits, hat);  // what forward dropped enters nothing, whatever it was
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            sum[kSums][e] = fma2(d[e], hat[e], sum[kSums][e]);
            d[e] = mul2(d[e], pa[e]);
          }
        }
      }
      store_columns<T, TPR, VEC>(pdb, c, cols, d);
      pdb += step * A.lddblock;
    }
    if (++stage == kStages) stage = 0;
  }
  copies_wait<0>();
  across.end();
  if (!A.part) return;
  // the upper half of the row groups hand their sums to the lower, until one has them
  constexpr int kPairs = kKinds * 4;
  f2* const join = reinterpret_cast<f2*>(dynamic);
#pragma unroll 1
  for (int n = kGroups; n > 1; n /= 2) {
    const int low = n / 2;
    __syncthreads();
    if (group >= low && group < n) {
#pragma unroll
      for (int i = 0; i < kPairs; ++i) join[((group - low) * kPairs + i) * TPR + threadIdx.x % TPR] = sum[i / 4][i % 4];
    }
    __syncthreads();
    if (group < low) {
#pragma unroll
      for (int i = 0; i < kPairs; ++i) sum[i / 4][i % 4] = add2(sum[i / 4][i % 4], join[(group * kPairs + i) * TPR + threadIdx.x % TPR]);
    }
  }
  if (group == 0 && c < cols) {
    float* p = A.part + (int64_t)(blockIdx.x / blocks) * 4 * cols + c;
#pragma unroll
    for (int k = 0; k < kKinds; ++k) store_group8<float, false>(p + (RMS ? 2 * k : k) * cols, cols - c, sum[k]);
  }
}
template <typename T, int TPR, bool VEC, int SIDE>
constexpr int kBackwardSmem = [] {
  constexpr int ring = RowStream<T, TPR, 1, VEC, 4, kBackwardStages<T, VEC>, kBackwardThreads>::kBytes, join = kBackwardThreads / 2 * (2 + SIDE) * 4 * 8;
  return ring > join ? ring : join;
}();

// ------------------------------------------------------------------------------------------------
// Rows wider than a cluster holds (65536 columns, backward 32768), read again for each step: one block a row, a thread eight columns at a
// time by single elements.  Right at any width, not fast: as the form for all rows it took 135 us where forward now takes 26.
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
static __global__ void __launch_bounds__(kWideThreads) k_rn_forward_wide(const ResidualForward A) {
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
  const ResidualBackward& A;
  const Generator& gen;
  int64_t r;
  float mean, rstd, block_mean, block_rstd;
  __device__ __forceinline__ RowBackward(const ResidualBackward& a, const Generator& g, int64_t row)
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
  // the block normalised, or without a norm behind it what stays of it: what forward dropped enters nothing, whatever it was
  __device__ __forceinline__ void bhat(int c, f2 (&b)[4]) const {
    load(A.block, A.ldblock, c, b);
    if (A.block_gamma) {
#pragma unroll
      for (int e = 0; e < 4; ++e) b[e] = mul2(add2(b[e], splat(-block_mean)), splat(block_rstd));
    } else if (gen.threshold) {
      gen.keep8(gen.draw(r * A.groups + c / 8), b);
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
static __global__ void __launch_bounds__(kWideThreads) k_rn_backward_wide(const ResidualBackward A) {
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
static __global__ void __launch_bounds__(kWideThreads) k_rn_param_wide(const ResidualBackward A, int64_t run) {
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

// The parameters' gradients from the four sums of each part, added in a fixed order: a block has eight columns (a sector of a
// part's row), an eighth of its threads to each of them.  Bound by latency: 1024 threads read 152 parts in two steps where every block has an SM,
// 256 in five where there are more (a call of 8192 x 2048: 47.9 us with 1024, 46.6 with 256; of 16384 x 1024: 36.5 and 38.3).
struct ParamGrads {
  void *dgamma, *dbeta, *dblock_gamma, *dblock_beta, *dgate;
};
template <typename G, int THREADS>
static __global__ void __launch_bounds__(THREADS) k_rn_params(const float* __restrict__ part, int64_t parts, int cols, const float* __restrict__ block_gamma,
                                                              const float* __restrict__ block_beta, const float* __restrict__ gate, const ParamGrads out) {
  constexpr int kRows = THREADS / 8;
  __shared__ float red[THREADS / 32][32];
  const int col = threadIdx.x & 7, row = threadIdx.x >> 3, c = blockIdx.x * 8 + col;
  const bool need[4] = {out.dgamma != nullptr, out.dbeta != nullptr, out.dblock_gamma || out.dgate, out.dblock_beta || (out.dgate && block_beta)};
  in_turn();
  float s[4] = {};
  if (c < cols) {
#pragma unroll 2
    for (int64_t p = row; p < parts; p += kRows) {
      const float* q = part + p * 4 * cols + c;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (need[k]) s[k] += q[(int64_t)k * cols];
    }
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    s[k] += __shfl_xor_sync(0xffffffffu, s[k], 8);
    s[k] += __shfl_xor_sync(0xffffffffu, s[k], 16);
  }
  red[warp][lane] = lane < 16 ? (lane < 8 ? s[0] : s[1]) : (lane < 24 ? s[2] : s[3]);  // eight columns of each kind
  __syncthreads();
  if (warp != 0) return;
  float total = 0.0f;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) total += red[w][lane];
  const float dbeta = __shfl_sync(0xffffffffu, total, 8 + col), a = __shfl_sync(0xffffffffu, total, 16 + col), b = __shfl_sync(0xffffffffu, total, 24 + col);
  if (lane >= 8 || c >= cols) return;
  const float at = gate ? gate[c] : 1.0f;
  if (out.dgamma) static_cast<G*>(out.dgamma)[c] = from_f<G>(total);
  if (out.dbeta) static_cast<G*>(out.dbeta)[c] = from_f<G>(dbeta);
  if (out.dblock_gamma) static_cast<G*>(out.dblock_gamma)[c] = from_f<G>(a * at);
  if (out.dblock_beta) static_cast<G*>(out.dblock_beta)[c] = from_f<G>(b * at);
  if (out.dgate) static_cast<G*>(out.dgate)[c] = from_f<G>(block_gamma ? fmaf(a, block_gamma[c], block_beta ? b * block_beta[c] : 0.0f) : a);
}

// ------------------------------------------------------------------------------------------------
// host side

inline unsigned at_most(int64_t want, int64_t per_sm) {
  const int64_t most = (int64_t)sm_count() * per_sm;
  return (unsigned)(want < most ? want : most);
}
// The blocks of a kernel that an SM holds at once, asked once for each device; `least` are what its launch bounds leave room for.
struct Held {
  std::atomic<int> blocks[64];
  template <typename Kernel>
  int operator()(Kernel* kernel, int threads, int bytes, int least) {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return least;
    if ((n = blocks[dev].load(std::memory_order_relaxed)) > 0) return n;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, bytes) != cudaSuccess || n < least)
      return least;
    blocks[dev].store(n, std::memory_order_relaxed);
    return n;
  }
};
// With `bytes` of dynamic shared memory, which a kernel is allowed once for each device, in clusters of `blocks`.
template <typename Args>
inline cudaError_t launch_rows(void (*kernel)(const Args), std::atomic<uint64_t>& ready, unsigned grid, int threads, int bytes, int blocks, cudaStream_t s,
                               const Args& a) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (!(ready.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid * (unsigned)blocks);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)bytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2]{};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)blocks;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = blocks > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

// the widest rows that one block holds in registers, up to eight of them as a cluster; wider ones are read again for each step
constexpr int kForwardCols = 512 * 2 * 8, kBackwardCols = 512 * 8;
inline int cluster_for(int64_t cols, int held) {
  int blocks = 1;
  while (cols > (int64_t)blocks * held) blocks *= 2;
  return blocks;
}

// f(threads a row): the fewest that hold `cols` columns, eight each
template <typename F>
auto with_threads(int64_t cols, F&& f) {
  using std::integral_constant;
  if (cols <= 64) return f(integral_constant<int, 8>{});
  if (cols <= 128) return f(integral_constant<int, 16>{});
  if (cols <= 256) return f(integral_constant<int, 32>{});
  if (cols <= 512) return f(integral_constant<int, 64>{});
  if (cols <= 1024) return f(integral_constant<int, 128>{});
  if (cols <= 2048) return f(integral_constant<int, 256>{});
  return f(integral_constant<int, 512>{});
}

template <typename T, int TPR, int CH, int NR, bool VEC, bool POST, bool CLUSTER>
cudaError_t run_forward(const ResidualForward& a, cudaStream_t s) {
  static std::atomic<uint64_t> ready{0};
  // As many blocks as the SMs hold, and no fewer: blocks come up while those of the kernel before leave, six to one SM then and four to another
  // where six fit and the grid has five for each (16384 x 1024 bf16 layer norm with dropout, two rows at a time: 25.5 us or 30 from one
  // call to the next).
  static Held held{};
  constexpr int kThreads = kForwardThreads<TPR>, kBytes = RowStream<T, TPR, CH, VEC, 2 * NR, kForwardStages<T>, kThreads, NR>::kBytes;
  const int blocks = CLUSTER ? cluster_for(a.cols, kForwardCols) : 1;
  const int64_t per_sm = held(k_rn_forward<T, TPR, CH, NR, VEC, POST, CLUSTER>, kThreads, kBytes, kForwardBlocks<TPR, CH, NR, POST>);
  const int64_t most = (int64_t)sm_count() * per_sm / blocks, want = ceil_div(a.rows, kForwardThreads<TPR> / TPR * NR);
  return launch_rows(k_rn_forward<T, TPR, CH, NR, VEC, POST, CLUSTER>, ready, (unsigned)(want < most ? want : most), kThreads, kBytes, blocks, s, a);
}
template <typename T>
cudaError_t rn_forward(ResidualForward a, cudaStream_t s) {
  if (a.cols > kForwardCols * kClusterMost) return launch_after(k_rn_forward_wide<T>, at_most(a.rows, 8), kWideThreads, s, a);
  auto on16 = [](const void* p, int64_t ld) { return aligned(p, 16) && (ld * (int64_t)sizeof(T)) % 16 == 0; };
  const bool vec = a.cols % 8 == 0 && on16(a.x, a.ldx) && on16(a.block, a.ldblock) && on16(a.s, a.lds) && on16(a.y, a.ldy);
  // Two rows at a time where there are enough for all SMs and it gains, with dropout or a norm behind the block (us for bf16, one and two,
  // medians over placements that differ by 1%: 16384 x 1024 with dropout, layer norm 28.7, 26.0, RMS norm 25.3, 23.4; layer norms on both sides
  // 30.9, 26.1, RMS norms 23.3, 23.0; 8192 x 2048 layer norm with dropout 30.7, 24.6).  Not where it does not, alone (layer norm 23.2, 23.3, RMS
  // norm 22.4, 22.2; 8192 x 2048 layer norm 23.3, 22.5).
  const bool two = a.drop.threshold || a.block_gamma;
  auto by = [&](auto tpr, auto ch, auto cluster) {
    constexpr int kTpr = decltype(tpr)::value, kCh = decltype(ch)::value;
    constexpr bool kCluster = decltype(cluster)::value;
    auto go = [&](auto post) {
      constexpr bool kPost = decltype(post)::value;
      if (!vec) return run_forward<T, kTpr, kCh, 1, false, kPost, kCluster>(a, s);
      if constexpr (sizeof(T) == 2 && kCh == 1 && !kCluster) {
        if (two && a.rows * kTpr >= (int64_t)sm_count() * 1280) return run_forward<T, kTpr, kCh, 2, true, kPost, kCluster>(a, s);
      }
      return run_forward<T, kTpr, kCh, 1, true, kPost, kCluster>(a, s);
    };
    return a.block_gamma ? go(std::true_type{}) : go(std::false_type{});
  };
  using std::integral_constant;
  using Two = integral_constant<int, 2>;
  if (a.cols > kForwardCols && !(a.status = status_word())) return cudaErrorUnknown;
  a.stall_tx = stall_bytes();
  if (a.cols > kForwardCols) return by(integral_constant<int, 512>{}, Two{}, std::true_type{});
  if (a.cols > 4096) return by(integral_constant<int, 512>{}, Two{}, std::false_type{});
  return with_threads(a.cols, [&](auto tpr) { return by(tpr, integral_constant<int, 1>{}, std::false_type{}); });
}

template <typename T, int TPR, bool VEC, int SIDE, bool CLUSTER, bool RMS>
cudaError_t run_backward(const ResidualBackward& a, unsigned parts, cudaStream_t s) {
  static std::atomic<uint64_t> ready{0};
  return launch_rows(k_rn_backward<T, TPR, VEC, SIDE, CLUSTER, RMS>, ready, parts, kBackwardThreads, kBackwardSmem<T, TPR, VEC, SIDE>,
                     CLUSTER ? cluster_for(a.cols, kBackwardCols) : 1, s, a);
}
// Takes the workspace; with `run`, enqueues the work too.
template <typename T>
cudaError_t rn_backward(ResidualBackward a, const ParamGrads& g, int32_t grad_dtype, char* workspace, int64_t* used, cudaStream_t s, bool run) {
  const bool params = g.dgamma || g.dbeta || g.dblock_gamma || g.dblock_beta || g.dgate, wide = a.cols > kBackwardCols * kClusterMost;
  const int64_t run_rows = a.rows ? ceil_div(a.rows, 64) : 1;  // of a wide kernel's part
  const int64_t parts = a.rows == 0 ? 0
                        : wide      ? ceil_div(a.rows, run_rows)
                        : a.cols > kBackwardCols ? std::min(a.rows, (int64_t)std::max(sm_count() / cluster_for(a.cols, kBackwardCols), 1))
                                    : with_threads(a.cols, [&](auto tpr) { return (int64_t)at_most(ceil_div(a.rows, kBackwardThreads / decltype(tpr)::value), 1); });
  const int64_t part_bytes = params ? (parts * 4 * a.cols * 4 + 15) & ~(int64_t)15 : 0;
  *used = part_bytes + (wide && a.gamma ? a.rows * 8 : 0);
  if (!run) return cudaSuccess;
  a.part = params ? reinterpret_cast<float*>(workspace) : nullptr;
  a.sums = reinterpret_cast<float*>(workspace + part_bytes);
  cudaError_t e = cudaSuccess;
  if (a.rows == 0) {
  } else if (wide) {
    e = launch_after(k_rn_backward_wide<T>, at_most(a.rows, 8), kWideThreads, s, a);
    if (e == cudaSuccess && params)
      e = launch_after(k_rn_param_wide<T>, dim3((unsigned)ceil_div(a.cols, kWideThreads * 8), (unsigned)parts), kWideThreads, s, a, run_rows);
  } else {
    auto on16 = [](const void* p, int64_t ld) { return aligned(p, 16) && (ld * (int64_t)sizeof(T)) % 16 == 0; };
    const bool vec = a.cols % 8 == 0 && on16(a.dy, a.lddy) && on16(a.ds, a.ldds) && on16(a.s, a.lds) && on16(a.block, a.ldblock) && on16(a.dx, a.lddx) &&
                     on16(a.dblock, a.lddblock);
    auto by = [&](auto tpr, auto cluster) {
      constexpr int kTpr = decltype(tpr)::value;
      constexpr bool kCluster = decltype(cluster)::value;
      auto go = [&](auto v, auto rms) {
        constexpr bool kVec = decltype(v)::value, kRms = decltype(rms)::value;
        if (a.block_gamma) return run_backward<T, kTpr, kVec, kBlockNorm, kCluster, kRms>(a, (unsigned)parts, s);
        return a.gate ? run_backward<T, kTpr, kVec, kBlockGate, kCluster, kRms>(a, (unsigned)parts, s)
                      : run_backward<T, kTpr, kVec, kBlockPlain, kCluster, kRms>(a, (unsigned)parts, s);
      };
      if (!vec) return go(std::false_type{}, std::false_type{});
      return a.layer ? go(std::true_type{}, std::false_type{}) : go(std::true_type{}, std::true_type{});
    };
    if (a.cols > kBackwardCols && !(a.status = status_word())) return cudaErrorUnknown;
    a.stall_tx = stall_bytes();
    e = a.cols > kBackwardCols ? by(std::integral_constant<int, 512>{}, std::true_type{}) : with_threads(a.cols, [&](auto tpr) { return by(tpr, std::false_type{}); });
  }
  if (e != cudaSuccess || !params) return e;
  auto finish = [&](auto g0) {
    using G = decltype(g0);
    const unsigned blocks = (unsigned)ceil_div(a.cols, 8);
    if ((int)blocks <= sm_count()) return launch_after(k_rn_params<G, 1024>, blocks, 1024, s, a.part, parts, a.cols, a.block_gamma, a.block_beta, a.gate, g);
    return launch_after(k_rn_params<G, 256>, blocks, 256, s, a.part, parts, a.cols, a.block_gamma, a.block_beta, a.gate, g);
  };
  return grad_dtype == ONEBIT_F32 ? finish(float{}) : grad_dtype == ONEBIT_F16 ? finish(__half{}) : finish(__nv_bfloat16{});
}

}  // namespace layers
}  // namespace onebit
