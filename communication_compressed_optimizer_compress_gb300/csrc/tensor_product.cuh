// tensor_product.cuh -- C[m][n] = sum_k A(m,k) B(n,k) of 16-bit operands on the tensor cores, accumulated
// in fp32, with an epilogue that turns the fp32 tile into what the caller stores.
//
// Each operand lies in memory with its contraction index contiguous ("K-major": A is m rows of k) or
// with its own index contiguous ("MN-major": A is k rows of m), which covers x w^T (K, K), dy w (K, MN)
// and dy^T x (MN, MN) without transposing anything.
//
// One block (or a pair of blocks on neighbouring SMs) computes a tile of 128 (256) rows by 128 (256)
// columns at a time.  Warp 0 copies operand slabs of 64 contraction elements into a ring of shared
// memory stages with TMA; warp 1 issues the tensor-core instructions; eight warps (a pair's block:
// sixteen) read finished accumulators out of tensor memory and run the epilogue.  Two accumulators alternate, so that the
// epilogue of one tile runs under the products of the next.  In a pair each block holds half of A's
// rows and half of B's, and the even block's instructions use both halves: each SM's shared memory
// then feeds a 256x256 tile with the traffic of a 128x128 one.
//
// Bound by the tensor cores where the epilogue is short (16384 x 4096 x 1024: 84 us, 1630 TFLOP/s of the 1878 measured
// for the library's products), by epilogue and tensor cores together with gelu and codes (16384 x 1024 x 4096 103 us, with
// gelu alone 90, where its 14 waves of tiles need 70 for the products by themselves), and by 64 bytes a clock into an SM where single
// blocks have a tile each (0.26 us a slab).
//
// A product without an activation epilogue (dw in any type, whose contraction is all tokens, and partial sums) is
// accumulated in chunks of kFoldSlabs slabs, whose sums the epilogue warps add up in registers: the tensor cores' own running
// sum loses about 2^-26 of its size a step (measured: 1.9e-6 of the result's norm after 2048 terms).
#pragma once

#include <cuda.h>  // CUtensorMap: types only, the encoder is looked up at run time

#include <atomic>

#include "layers_common.cuh"

namespace onebit {
namespace layers {

constexpr int kSlabK = 64;                    // contraction elements per stage: 128 bytes, one swizzle row
constexpr int kRowsPerBlock = 128;            // rows of each operand that a block holds
constexpr int kOperandBytes = kRowsPerBlock * kSlabK * 2;
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kStages = 5;
template <int CTAS>
constexpr int kEpilogueWarps = 8 * CTAS;      // 128 rows are 4 quarters of the tensor memory; 64 columns a warp
template <int CTAS>
constexpr int kProductThreads = 128 + 32 * kEpilogueWarps<CTAS>;
// A pair's block is launched with 640 * 96 registers; 128 * 56 + 512 * 104 of them are used.
constexpr int kControlRegs = 56, kEpilogueRegs = 104;
// A warp's staging buffer: 32 rows of 64 bytes (2048, swizzled, what TMA stores; padded to 80 bytes a row
// where single elements are stored), behind it 32 rows of 32 codes, and 64 columns' bias.
constexpr int kStagingRow = 80;
constexpr int kCodeStaging = 32 * kStagingRow;
constexpr int kBiasStaging = kCodeStaging + 1024;
constexpr int kStagingBytes = kBiasStaging + 512;
constexpr int kBarrierBytes = 256;
template <int CTAS>
constexpr int kProductSmem = 1024 + kStages * kStageBytes + kEpilogueWarps<CTAS> * kStagingBytes + kBarrierBytes + kActConsts * 8;
static_assert(kStagingBytes % 512 == 0, "the swizzle's period");
constexpr int kFoldSlabs = 8;                 // slabs that an accumulator of a folded product sums up
constexpr int kGroupTiles = 8;                // tile rows that are walked together, for the L2

constexpr unsigned kStatusGaveUp = 1u;

struct ProductArgs {
  CUtensorMap a, b;
  int64_t m;
  int32_t n;
  int32_t slabs;             // of the whole contraction
  int32_t tiles_m, tiles_n;
  int32_t splits, split_slabs;
  uint32_t units;            // tiles times splits
  uint32_t group_mul, group_shift;  // reciprocal of the tiles in a group of kGroupTiles tile rows
  uint32_t idesc;
  uint32_t stall_tx;         // test hook: bytes that every stage waits for and no copy brings (normally 0)
  unsigned int* status;
};

// ------------------------------------------------------------------------------------------------
// PTX

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// What this arrival announces is that loads from tensor memory are done, which tcgen05.wait has seen to: no
// memory has to be released with it.
__device__ __forceinline__ void bar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Address of this block's shared memory word `addr` in the block `rank` of the cluster.
__device__ __forceinline__ uint32_t in_block(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// One box of a matrix into this block's shared memory; `bar` may be the other block's of a pair.
template <int CTAS>
__device__ __forceinline__ void copy_box(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, uint32_t bar) {
  if (CTAS == 2)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst), "l"(map),
        "r"(x), "r"(y), "r"(bar)
        : "memory");
}

template <int CTAS>
__device__ __forceinline__ void tmem_alloc(uint32_t dst, uint32_t cols) {
  if (CTAS == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
}
template <int CTAS>
__device__ __forceinline__ void tmem_free(uint32_t base, uint32_t cols) {
  if (CTAS == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols) : "memory");
  else
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols) : "memory");
}
// The barrier (of both blocks of a pair) is arrived at when this thread's instructions so far are done.
template <int CTAS>
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  if (CTAS == 2)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar), "h"((uint16_t)3)
        : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// 16 columns, for the folding sums
__device__ __forceinline__ void tmem_load16(uint32_t addr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(addr));
}
__device__ __forceinline__ void tmem_hold16(float* v) {
  asm volatile("" : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]));
}
// Waits for this warp's loads.  The values pass through the statement, so that nothing that uses them
// can be moved ahead of it.
__device__ __forceinline__ void tmem_hold32(float* v) {
  asm volatile("" : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31]));
}
__device__ __forceinline__ void tmem_wait_load() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// 32 columns of the 32 lanes that this warp may read, as fp32 pairs
__device__ __forceinline__ void tmem_load32(uint32_t addr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, "
      "%29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]),
        "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
        "=r"(r[31])
      : "r"(addr));
}

// Shared-memory matrix descriptor: 128-byte swizzle over groups of 8 rows of 128 bytes (1024 bytes).
// K-major: a row is one m (n) with 64 k; groups of 8 m follow each other (stride 1024), and a step of
// 16 k is 32 bytes along the row.  MN-major: a row is one k with 64 m; groups of 8 k follow each other
// (stride 1024), the next 64 m lie one 64-row box (8192 bytes) further, and a step of 16 k is 2048 bytes.
// The low word holds the address and the leading stride, the high word is the same for all.
template <bool MN>
__device__ __forceinline__ uint32_t operand_desc(uint32_t addr) {
  return (addr >> 4 & 0x3fff) | (MN ? 8192u >> 4 : 1u) << 16;
}
constexpr uint32_t kDescHigh = (1024 >> 4) | 1u << 14 | 2u << 29;
template <bool MN>
constexpr uint32_t kStep16 = MN ? 2048 >> 4 : 32 >> 4;

// The products of one slab: four steps of 16.  The thread that issues them has about 500 clocks a slab
// before the tensor cores run dry, beside four busy warps of its scheduler, so the loop around this is kept
// to a few instructions.
template <int CTAS, bool A_MN, bool B_MN>
__device__ __forceinline__ void mma_slab(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
#pragma unroll
  for (int q = 0; q < kSlabK / 16; ++q) {
    if (CTAS == 2)
      asm volatile(
          "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.u32 p, %4, 0;\n\tmov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
          "tcgen05.mma.cta_group::2.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
          "r"(a + q * kStep16<A_MN>), "r"(b + q * kStep16<B_MN>), "r"(idesc), "r"((uint32_t)(add || q > 0)), "r"(kDescHigh)
          : "memory");
    else
      asm volatile(
          "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.u32 p, %4, 0;\n\tmov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
          "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
          "r"(a + q * kStep16<A_MN>), "r"(b + q * kStep16<B_MN>), "r"(idesc), "r"((uint32_t)(add || q > 0)), "r"(kDescHigh)
          : "memory");
  }
}

// ------------------------------------------------------------------------------------------------
// Waits end after about a second: the block's flag is set, every other wait of the block ends too, and
// the status word says so.
struct Wait {
  volatile int* gave_up;
  unsigned int* status;
  __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const {
    if (bar_try(bar, parity)) return true;
    const long long t0 = clock64();
    while (!bar_try(bar, parity)) {
      if (*gave_up) return false;
      if (clock64() - t0 > 2000000000ll) {
        *gave_up = 1;
        atomicOr(status, kStatusGaveUp);
        return false;
      }
    }
    return true;
  }
};

// ------------------------------------------------------------------------------------------------
// Rows of 64 bytes between registers (a lane has a row) and memory (four lanes share a row, so that every
// access is whole sectors), through the warp's staging buffer.

// Before a staging buffer is written again: the warp's stores out of it have read it.
__device__ __forceinline__ void staging_free() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  __syncwarp();
}
// A staged box to a matrix, by one lane; what lies outside the matrix is left out.
__device__ __forceinline__ void copy_out(const CUtensorMap* map, uint32_t src, int32_t x, int32_t y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map), "r"(x), "r"(y), "r"(src) : "memory");
}
__device__ __forceinline__ void store_box(const CUtensorMap* map, uint32_t src, int32_t x, int32_t y) {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
  if ((threadIdx.x & 31) == 0) {
    copy_out(map, src, x, y);
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
}

// A matrix that an epilogue writes: by TMA where its rows start on 16 bytes, element by element elsewhere.
template <typename T>
struct Output {
  CUtensorMap map;
  T* p;
  int64_t ld;
  bool by_tma;
};

template <typename T>
__device__ __forceinline__ void stage_rows(char* staging, const uint32_t (&v)[16]) {
  const int lane = threadIdx.x & 31, swap = lane >> 1 & 3;  // 64-byte swizzle: 16-byte chunk j of row r lies at j ^ (r / 2 % 4)
#pragma unroll
  for (int j = 0; j < 4; ++j)
    *reinterpret_cast<uint4*>(staging + lane * 64 + (j ^ swap) * 16) = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
}
__device__ __forceinline__ void stage_codes(char* staging, const uint32_t (&v)[8]) {
  const int lane = threadIdx.x & 31, swap = lane >> 2 & 1;  // 32-byte swizzle: chunk j of row r lies at j ^ (r / 4 % 2)
#pragma unroll
  for (int j = 0; j < 2; ++j)
    *reinterpret_cast<uint4*>(staging + kCodeStaging + lane * 32 + (j ^ swap) * 16) = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
}

// 64 bytes of a lane's row.  (With ordinary stores the way through shared memory and back to registers
// took most of an epilogue's time, as it shares the SM's shared-memory bandwidth with the products.)
template <typename T>
__device__ __forceinline__ void store_rows(char* staging, const uint32_t (&v)[16], const Output<T>& out, int64_t row0, int64_t rows, int col0, int cols) {
  constexpr int kCols = 64 / sizeof(T);
  const int lane = threadIdx.x & 31;
  staging_free();
  if (out.by_tma) {
    stage_rows<T>(staging, v);
    store_box(&out.map, smem_addr(staging), col0, (int32_t)row0);
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    *reinterpret_cast<uint4*>(staging + lane * kStagingRow + j * 16) = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
  __syncwarp();
  constexpr int kPer = 32 / kCols;  // rows at a time
  const int q = lane % kCols, r0 = lane / kCols;
  T* p = out.p + (row0 + r0) * out.ld + col0 + q;
  const int last = col0 + q < cols && row0 < rows ? (int)(rows - row0 < 32 ? rows - row0 : 32) : 0;
#pragma unroll 1
  for (int i = 0; i < 32; i += 16 * kPer) {  // sixteen reads at a time, then their stores (one by one: 22.6 us for 18.3)
    T t[16];
#pragma unroll
    for (int k = 0; k < 16; ++k)
      t[k] = reinterpret_cast<const T*>(staging + (i + k * kPer + r0) * kStagingRow)[q];
#pragma unroll
    for (int k = 0; k < 16; ++k, p += kPer * out.ld)
      if (i + k * kPer + r0 < last) *p = t[k];
  }
  __syncwarp();
}

// A matrix that an epilogue reads.  Where its rows start on 32 bytes a lane reads its own row, whole sectors at a
// time, half of its 64 columns ahead: the first before the product is waited for, the second under the first
// one's arithmetic (16384 x 1024 x 4096 through gelu' from codes: 117 us, 128 through the staging buffer).
template <typename T>
struct Input16 {
  const T* p;
  int64_t ld;
  bool wide;   // rows on 32 bytes
  bool vec;    // rows on 16 bytes

  __device__ __forceinline__ bool ahead(int64_t row, int64_t rows, int col0, int cols, uint32_t (&v)[16]) const {
    if (!wide || col0 + 32 > cols) return false;
    if (row < rows) {
      load32(p + row * ld + col0, v);
      load32(p + row * ld + col0 + 16, v + 8);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = 0;
    }
    return true;
  }
};

// 32 columns of a 16-bit matrix to the staging buffer, and from there a lane's row
template <typename T>
__device__ __forceinline__ void fetch_rows(char* staging, const T* p, int64_t ld, int64_t row0, int64_t rows, int col0, int cols, bool vec) {
  const int lane = threadIdx.x & 31;
  staging_free();
  if (vec && (col0 + 32 <= cols || cols % 8 == 0)) {
    const int c = col0 + (lane & 3) * 8;
    const T* q = p + (row0 + (lane >> 2)) * ld + c;
    uint4 t[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      t[i] = row0 + i * 8 + (lane >> 2) < rows && c < cols ? *reinterpret_cast<const uint4*>(q + i * 8 * ld) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(staging + (i * 8 + (lane >> 2)) * kStagingRow + (lane & 3) * 16) = t[i];
  } else {
    for (int r0 = 0; r0 < 32; r0 += 16) {  // sixteen loads in flight
      T t[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) t[i] = row0 + r0 + i < rows && col0 + lane < cols ? p[(row0 + r0 + i) * ld + col0 + lane] : from_f<T>(0.0f);
#pragma unroll
      for (int i = 0; i < 16; ++i) reinterpret_cast<T*>(staging + (r0 + i) * kStagingRow)[lane] = t[i];
    }
  }
  __syncwarp();
}
__device__ __forceinline__ void take_rows(const char* staging, uint32_t (&v)[16]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint4 t = *reinterpret_cast<const uint4*>(staging + lane * kStagingRow + j * 16);
    v[4 * j] = t.x, v[4 * j + 1] = t.y, v[4 * j + 2] = t.z, v[4 * j + 3] = t.w;
  }
  __syncwarp();
}

template <typename T>
__device__ __forceinline__ void load_rows(char* staging, uint32_t (&v)[16], const T* p, int64_t ld, int64_t row0, int64_t rows, int col0, int cols,
                                          bool vec) {
  fetch_rows(staging, p, ld, row0, rows, col0, cols, vec);
  take_rows(staging, v);
}

// 32 codes of a row, packed in 8 words; codes are contiguous rows of `cols`
constexpr int kCodeRow = 48;
__device__ __forceinline__ void store_codes(char* staging, const uint32_t (&v)[8], const Output<int8_t>& out, int64_t row0, int64_t rows, int col0, int cols) {
  const int lane = threadIdx.x & 31;
  staging_free();
  if (out.by_tma) {
    stage_codes(staging, v);
    store_box(&out.map, smem_addr(staging + kCodeStaging), col0, (int32_t)row0);
    return;
  }
#pragma unroll
  for (int j = 0; j < 2; ++j)
    *reinterpret_cast<uint4*>(staging + lane * kCodeRow + j * 16) = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
  __syncwarp();
  int8_t* p = out.p + row0 * cols + col0 + lane;
  const int last = col0 + lane < cols && row0 < rows ? (int)(rows - row0 < 32 ? rows - row0 : 32) : 0;
#pragma unroll 1
  for (int i = 0; i < 32; i += 16) {
    int8_t t[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) t[k] = (staging + (i + k) * kCodeRow)[lane];
#pragma unroll
    for (int k = 0; k < 16; ++k, p += cols)
      if (i + k < last) *p = t[k];
  }
  __syncwarp();
}
// y and the codes of 32 columns with one fence between their staging and their copies
template <typename T>
__device__ __forceinline__ void store_rows_and_codes(char* staging, const uint32_t (&v)[16], const Output<T>& y, const uint32_t (&c)[8],
                                                     const Output<int8_t>& codes, int64_t row0, int64_t rows, int col0, int cols) {
  if (y.by_tma && codes.by_tma) {
    staging_free();
    stage_rows<T>(staging, v);
    stage_codes(staging, c);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if ((threadIdx.x & 31) == 0) {
      copy_out(&y.map, smem_addr(staging), col0, (int32_t)row0);
      copy_out(&codes.map, smem_addr(staging + kCodeStaging), col0, (int32_t)row0);
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
    return;
  }
  store_codes(staging, c, codes, row0, rows, col0, cols);
  store_rows(staging, v, y, row0, rows, col0, cols);
}
__device__ __forceinline__ void fetch_codes(char* staging, const int8_t* p, int64_t row0, int64_t rows, int col0, int cols, bool vec) {
  const int lane = threadIdx.x & 31;
  staging_free();
  if (vec) {
    const int c = col0 + (lane & 1) * 16;
    uint4 t[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = i * 16 + (lane >> 1);
      t[i] = row0 + r < rows && c < cols ? *reinterpret_cast<const uint4*>(p + (row0 + r) * cols + c) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) *reinterpret_cast<uint4*>(staging + (i * 16 + (lane >> 1)) * kCodeRow + (lane & 1) * 16) = t[i];
  } else {
    for (int r0 = 0; r0 < 32; r0 += 16) {
      int8_t t[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) t[i] = row0 + r0 + i < rows && col0 + lane < cols ? p[(row0 + r0 + i) * cols + col0 + lane] : (int8_t)0;
#pragma unroll
      for (int i = 0; i < 16; ++i) (staging + (r0 + i) * kCodeRow)[lane] = t[i];
    }
  }
  __syncwarp();
}
__device__ __forceinline__ void take_codes(const char* staging, uint32_t (&v)[8]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint4 t = *reinterpret_cast<const uint4*>(staging + lane * kCodeRow + j * 16);
    v[4 * j] = t.x, v[4 * j + 1] = t.y, v[4 * j + 2] = t.z, v[4 * j + 3] = t.w;
  }
  __syncwarp();
}

__device__ __forceinline__ void load_codes(char* staging, uint32_t (&v)[8], const int8_t* p, int64_t row0, int64_t rows, int col0, int cols, bool vec) {
  fetch_codes(staging, p, row0, rows, col0, cols, vec);
  take_codes(staging, v);
}

// ------------------------------------------------------------------------------------------------
// Epilogues.  A lane has row row0 + lane.  run() of the fused ones reads the warp's 64 columns from col0 on
// out of tensor memory, 32 at a time, by load(half, pairs), and calls release() after the last read: a rolled
// loop over the halves, with few registers and little code, lets sixteen warps run side by side.  (Eight warps of
// 232 registers that hold all 64 columns are no faster: 8.4 us a pair's tile of 1024 terms with gelu and checkpoint
// for 8.5, and 9.4 for 9.1 in the input's gradient.)

// The activation's constants, read once for 32 columns (volatile: as literals, or kept longer than that, they
// cost more registers or instructions than these few loads).
template <int ACT>
__device__ __forceinline__ ActConsts shared_consts(const f2* consts) {
  ActConsts k;
  if (ACT == ONEBIT_ACT_GELU || ACT == ONEBIT_ACT_GELU_TANH) {
#pragma unroll
    for (int i = 0; i < kActConsts; i += 2)
      asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(k.k[i]), "=l"(k.k[i + 1]) : "r"(smem_addr(consts + i)));
  }
  return k;
}

// The activation, and what the kept value is, are template parameters of the epilogues of pairs: with them
// decided at run time inside the loop the register allocation of the alternatives met in copies, 100 to 300 of
// a unit's 700 to 1700 instructions.  kAny decides at run time: the single blocks of small products, and in pairs a
// residual together with an activation or a checkpoint (16384 x 1024 x 4096 with gelu, residual and checkpoint 130 us,
// without the residual, in its own form, 103; 88 bytes of its registers spill).
constexpr int kAny = -1;
enum Kept16 { kKeptNone = 0, kKeptValue = 1, kKeptCodes = 2 };

template <typename T, int ACT, int CK, int RES>
struct ForwardEpilogue {
  // y = act(d + bias) + residual, and the 8-bit checkpoint of d + bias
  static constexpr bool kFold = false;
  const float* bias;
  Input16<T> residual;
  Output<T> y;
  Output<int8_t> codes;
  float* scales;  // NULL: no checkpoint
  int blocks;
  int act;

  __device__ __forceinline__ bool keeps() const { return CK == kAny ? scales != nullptr : CK == 1; }
  __device__ __forceinline__ bool adds() const { return RES == kAny ? residual.p != nullptr : RES == 1; }
  struct Ahead {};
  // before the product is waited for: the warp's 64 columns of the bias, two a lane (without one: zeros, as adding
  // them is cheaper than both ways meeting behind a branch), and the residual's first 32 to the staging buffer
  // (1237 x 1001 x 777 in odd rows: 18.3 -> 16.3 us with the setup beside the realigning kernel; ahead in registers it
  // is no faster: 16384 x 4096 x 1024 98.9 us for 98.1)
  __device__ __forceinline__ void prepare(Ahead&, int64_t row0, int64_t rows, int col0, int cols, char* staging) const {
    const int c = col0 + 2 * (threadIdx.x & 31);
    f2 b = 0;
    if (bias) b = pair(c < cols ? __ldg(bias + c) : 0.0f, c + 1 < cols ? __ldg(bias + c + 1) : 0.0f);
    reinterpret_cast<f2*>(staging + kBiasStaging)[threadIdx.x & 31] = b;
    __syncwarp();
    if (adds()) fetch_rows(staging, residual.p, residual.ld, row0, rows, col0, cols, residual.vec);
  }
  __device__ __forceinline__ void add_bias(f2 (&z)[16], int half, const char* staging) const {
    const ulonglong2* b = reinterpret_cast<const ulonglong2*>(staging + kBiasStaging + 128 * half);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const ulonglong2 v = b[i];
      z[2 * i] = add2(z[2 * i], v.x), z[2 * i + 1] = add2(z[2 * i + 1], v.y);
    }
  }
  template <int A>
  __device__ __forceinline__ void finish(const f2* consts, f2 (&z)[16], uint32_t (&v)[16]) const {  // v: in the residual, out y
    const ActConsts k = shared_consts<A>(consts);
    if (adds()) {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = narrow<T>(add2(act2<A>(k, z[i]), widen<T>(v[i])));
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = narrow<T>(act2<A>(k, z[i]));
    }
  }
  template <class Load, class Release>
  __device__ __forceinline__ void run(Ahead&, Load&& load, Release&& release, const f2* consts, int64_t row0, int64_t rows, int col0,
                                      int cols, char* staging) const {
    float inv = 0.0f;
    bool plain = true;  // no value of the warp's blocks is infinite or NaN
    if (keeps()) {  // columns past the end have z = 0: their operand rows were filled with zeros
      float most = 0.0f;
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        f2 z[16];
        load(half, z);
        add_bias(z, half, staging);
#pragma unroll
        for (int i = 0; i < 16; ++i) most = max_abs(most, z[i]);
      }
      const BlockScale s = block_scale(most);
      const int64_t row = row0 + (threadIdx.x & 31);
      if (row < rows) scales[row * blocks + col0 / kBlock] = s.scale;
      inv = s.inv;
      plain = __all_sync(0xffffffffu, s.scale == s.scale);
    }
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
      f2 z[16];
      uint32_t v[16], c[8];
      load(half, z);
      if (half) release();
      const int c0 = col0 + 32 * half;
      if (c0 >= cols) continue;
      add_bias(z, half, staging);
      if (keeps()) {
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = codes4_finite(z[2 * i], z[2 * i + 1], inv);
        if (!plain && inv == 0.0f) {
#pragma unroll
          for (int i = 0; i < 8; ++i) c[i] = 0;
        }
      }
      if (adds()) {
        if (!half) take_rows(staging, v);
        else load_rows(staging, v, residual.p, residual.ld, row0, rows, c0, cols, residual.vec);
      }
      if constexpr (ACT != kAny) finish<ACT>(consts, z, v);
      else if (act == ONEBIT_ACT_NONE) finish<ONEBIT_ACT_NONE>(consts, z, v);
      else if (act == ONEBIT_ACT_RELU) finish<ONEBIT_ACT_RELU>(consts, z, v);
      else if (act == ONEBIT_ACT_GELU) finish<ONEBIT_ACT_GELU>(consts, z, v);
      else finish<ONEBIT_ACT_GELU_TANH>(consts, z, v);
      if (keeps()) store_rows_and_codes(staging, v, y, c, codes, row0, rows, c0, cols);
      else store_rows(staging, v, y, row0, rows, c0, cols);
    }
    __syncwarp();  // the bias has been read: prepare() may write the next
  }
};

template <typename T, int ACT, int KEPT>
struct InputGradEpilogue {
  // dx = d * act'(v) [+ add], and h = act(v) for the product of dw
  static constexpr bool kFold = false;
  Input16<T> x;          // the value before the activation,
  const int8_t* codes;   // or its checkpoint
  const float* scales;
  int blocks;
  Input16<T> add;
  Output<T> dx, h;  // h.p NULL: not wanted
  int act;
  int kept;         // Kept16: what is needed
  bool wide_codes, vec_codes;

  static constexpr bool kAheadCodes = KEPT == kKeptCodes, kAheadRow = KEPT == kKeptValue || KEPT == kKeptNone;
  static constexpr bool kStaged = KEPT == kAny;  // what is read first lies in the staging buffer ahead
  struct Ahead {
    uint32_t c[kAheadCodes ? 8 : 1];
    uint32_t v[kAheadRow ? 16 : 1];  // x, or add where x is not needed
  };
  __device__ __forceinline__ void fetch(Ahead& a, int64_t row, int64_t rows, int c0, int cols) const {
    if constexpr (kAheadCodes) {
      if (wide_codes && c0 + 32 <= cols && row < rows) load32(codes + row * cols + c0, a.c);
    }
    if constexpr (KEPT == kKeptValue) x.ahead(row, rows, c0, cols, a.v);
    if constexpr (KEPT == kKeptNone) {
      if (add.p) add.ahead(row, rows, c0, cols, a.v);
    }
  }
  __device__ __forceinline__ void prepare(Ahead& a, int64_t row0, int64_t rows, int col0, int cols, char* staging) const {
    if constexpr (!kStaged) fetch(a, row0 + (threadIdx.x & 31), rows, col0, cols);
    else if (kept == kKeptCodes) fetch_codes(staging, codes, row0, rows, col0, cols, vec_codes);
    else if (kept == kKeptValue) fetch_rows(staging, x.p, x.ld, row0, rows, col0, cols, x.vec);
    else if (add.p) fetch_rows(staging, add.p, add.ld, row0, rows, col0, cols, add.vec);
  }
  // z: the kept values; d: times the slope; v: out h
  template <int A>
  __device__ __forceinline__ void slopes(const ActConsts& k, f2 z, f2& d, uint32_t& v) const {
    f2 a, s;
    activate<A, true, A != ONEBIT_ACT_NONE>(k, z, a, s);
    if (A != ONEBIT_ACT_NONE) d = mul2(d, s);
    v = narrow<T>(a);
  }
  template <int A>
  __device__ __forceinline__ void by_value(const f2* consts, f2 (&d)[16], uint32_t (&v)[16]) const {
    const ActConsts k = shared_consts<A>(consts);
#pragma unroll
    for (int i = 0; i < 16; ++i) slopes<A>(k, widen<T>(v[i]), d[i], v[i]);
  }
  template <int A>
  __device__ __forceinline__ void by_codes(const f2* consts, f2 (&d)[16], const uint32_t (&c)[8], float scale, uint32_t (&v)[16]) const {
    const ActConsts k = shared_consts<A>(consts);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      f2 z[2];
      values4<T>(c[i], scale, z);
      slopes<A>(k, z[0], d[2 * i], v[2 * i]);
      slopes<A>(k, z[1], d[2 * i + 1], v[2 * i + 1]);
    }
  }
  template <class Load, class Release>
  __device__ __forceinline__ void run(Ahead& ahead, Load&& load, Release&& release, const f2* consts, int64_t row0, int64_t rows, int col0,
                                      int cols, char* staging) const {
    const int64_t row = row0 + (threadIdx.x & 31);
    const int need = KEPT == kAny ? kept : KEPT;
    float scale = 0.0f;
    if (need == kKeptCodes && row < rows) scale = __ldg(scales + row * blocks + col0 / kBlock);
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
      const int c0 = col0 + 32 * half;
      f2 d[16];
      uint32_t v[16];
      load(half, d);
      if (half) release();
      if (c0 >= cols) continue;
      const bool whole = c0 + 32 <= cols;
      if (need == kKeptCodes) {
        uint32_t c[8];
        if (kAheadCodes && wide_codes && whole) {
#pragma unroll
          for (int i = 0; i < 8; ++i) c[i] = ahead.c[kAheadCodes ? i : 0];
        } else if (kStaged && !half) {
          take_codes(staging, c);
        } else {
          load_codes(staging, c, codes, row0, rows, c0, cols, vec_codes);
        }
        if constexpr (kAheadCodes) {
          if (!half) fetch(ahead, row, rows, c0 + 32, cols);
        }
        if constexpr (ACT != kAny) by_codes<ACT>(consts, d, c, scale, v);
        else if (act == ONEBIT_ACT_NONE) by_codes<ONEBIT_ACT_NONE>(consts, d, c, scale, v);
        else if (act == ONEBIT_ACT_RELU) by_codes<ONEBIT_ACT_RELU>(consts, d, c, scale, v);
        else if (act == ONEBIT_ACT_GELU) by_codes<ONEBIT_ACT_GELU>(consts, d, c, scale, v);
        else by_codes<ONEBIT_ACT_GELU_TANH>(consts, d, c, scale, v);
      } else if (need == kKeptValue) {
        if (KEPT == kKeptValue && x.wide && whole) {
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = ahead.v[kAheadRow ? i : 0];
        } else if (kStaged && !half) {
          take_rows(staging, v);
        } else {
          load_rows(staging, v, x.p, x.ld, row0, rows, c0, cols, x.vec);
        }
        if constexpr (KEPT == kKeptValue) {
          if (!half) fetch(ahead, row, rows, c0 + 32, cols);
        }
        if constexpr (ACT != kAny) by_value<ACT>(consts, d, v);
        else if (act == ONEBIT_ACT_RELU) by_value<ONEBIT_ACT_RELU>(consts, d, v);
        else if (act == ONEBIT_ACT_GELU) by_value<ONEBIT_ACT_GELU>(consts, d, v);
        else by_value<ONEBIT_ACT_GELU_TANH>(consts, d, v);
      }
      if (need != kKeptNone && h.p) store_rows(staging, v, h, row0, rows, c0, cols);
      if (add.p) {
        if (KEPT == kKeptNone && add.wide && whole) {
#pragma unroll
          for (int i = 0; i < 16; ++i) d[i] = add2(d[i], widen<T>(ahead.v[kAheadRow ? i : 0]));
          if constexpr (KEPT == kKeptNone) {
            if (!half) fetch(ahead, row, rows, c0 + 32, cols);
          }
        } else {
          if (kStaged && !half && need == kKeptNone) take_rows(staging, v);
          else load_rows(staging, v, add.p, add.ld, row0, rows, c0, cols, add.vec);
#pragma unroll
          for (int i = 0; i < 16; ++i) d[i] = add2(d[i], widen<T>(v[i]));
        }
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = narrow<T>(d[i]);
      store_rows(staging, v, dx, row0, rows, c0, cols);
    }
  }
};

template <typename G>
struct PlainEpilogue {
  // the product itself in G; split s of a cut contraction goes to rows s * split_rows and on
  static constexpr bool kFold = true;
  static constexpr int act = ONEBIT_ACT_NONE;
  Output<G> out;
  int64_t split_rows;
  __device__ __forceinline__ void run(f2 (&d)[16], int64_t row0, int64_t rows, int col0, int cols, int split, char* staging) const {
    // a split's rows past its own end would fall into the next one's
    const int64_t at = row0 + split * split_rows, end = split * split_rows + rows;
    uint32_t v[16];
    if (sizeof(G) == 4) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 f = halves(d[8 * q + i]);
          v[2 * i] = __float_as_uint(f.x), v[2 * i + 1] = __float_as_uint(f.y);
        }
        if (col0 + 16 * q < cols) store_rows(staging, v, out, at, end, col0 + 16 * q, cols);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = narrow<std::conditional_t<sizeof(G) == 4, __half, G>>(d[i]);
      store_rows(staging, v, out, at, end, col0, cols);
    }
  }
};

// ------------------------------------------------------------------------------------------------

struct Tile {
  int64_t m0;
  int n0, split, first, slabs;
};
__device__ __forceinline__ int slabs_of(const ProductArgs& P, int split) {
  const int left = P.slabs - split * P.split_slabs;
  return left < P.split_slabs ? left : P.split_slabs;
}
template <int CTAS>
__device__ __forceinline__ Tile tile_of(const ProductArgs& P, uint32_t unit) {
  constexpr int kM = kRowsPerBlock * CTAS, kN = kRowsPerBlock * CTAS;
  Tile t;
  const uint32_t tile = P.splits == 1 ? unit : unit / P.splits;
  t.split = (int)(unit - tile * P.splits);
  // kGroupTiles tile rows side by side, column after column: the tiles in flight share operand slabs in L2.
  // The division by a group's tiles is a multiplication by its rounded-up reciprocal (exact below 2^31).
  const uint32_t g = (__umulhi(tile, P.group_mul) + tile) >> P.group_shift, m = g * kGroupTiles;
  const uint32_t in = tile - m * P.tiles_n, left = P.tiles_m - m;
  const uint32_t col = left >= kGroupTiles ? in / kGroupTiles : in / left, rows = left >= kGroupTiles ? kGroupTiles : left;
  t.m0 = (int64_t)(m + in - col * rows) * kM;
  t.n0 = (int)col * kN;
  t.first = t.split * P.split_slabs;
  t.slabs = slabs_of(P, t.split);
  return t;
}

template <int CTAS, bool A_MN, bool B_MN, class Epilogue>
__global__ void __launch_bounds__(kProductThreads<CTAS>, 1) k_product(const __grid_constant__ ProductArgs P, const __grid_constant__ Epilogue E) {
  constexpr int kTileN = kRowsPerBlock * CTAS;
  constexpr uint32_t kTmemCols = 2 * kTileN;    // two accumulators
  extern __shared__ char smem_raw[];
  // (an offset, not a rounded pointer: the compiler has to see that this is shared memory)
  char* smem = smem_raw + (-(int)smem_addr(smem_raw) & 1023);
  char* staging_base = smem + kStages * kStageBytes;
  char* bars = staging_base + kEpilogueWarps<CTAS> * kStagingBytes;
  f2* consts = reinterpret_cast<f2*>(bars + kBarrierBytes);  // on 16 bytes
  const uint32_t bar0 = smem_addr(bars);
  auto full = [&](int s) { return bar0 + 8 * s; };
  auto empty = [&](int s) { return bar0 + 8 * (kStages + s); };
  auto acc_full = [&](int s) { return bar0 + 8 * (2 * kStages + s); };
  auto acc_empty = [&](int s) { return bar0 + 8 * (2 * kStages + 2 + s); };
  const uint32_t drained = bar0 + 8 * (2 * kStages + 4);
  volatile uint32_t* tmem_ptr = reinterpret_cast<volatile uint32_t*>(bars + 8 * (2 * kStages + 5));
  volatile int* gave_up = reinterpret_cast<volatile int*>(bars + 8 * (2 * kStages + 6));

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CTAS == 2 ? cluster_rank() : 0;
  const uint32_t units = P.units, first_unit = blockIdx.x / CTAS, unit_step = gridDim.x / CTAS;
  const Wait wait{gave_up, P.status};

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) bar_init(full(s), 1), bar_init(empty(s), 1);
    for (int s = 0; s < 2; ++s) bar_init(acc_full(s), 1), bar_init(acc_empty(s), CTAS * kEpilogueWarps<CTAS>);
    bar_init(drained, 1);
    *gave_up = 0;
#pragma unroll
    for (int i = 0; i < kActConsts; ++i)
      consts[i] = splat(E.act == ONEBIT_ACT_GELU ? act_const(ONEBIT_ACT_GELU, i) : act_const(ONEBIT_ACT_GELU_TANH, i));
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc<CTAS>(smem_addr((const void*)tmem_ptr), kTmemCols);
  tmem_fence_before();
  __syncthreads();
  if (CTAS == 2) cluster_sync();  // the other block's barriers are ready too
  tmem_fence_after();
  const uint32_t tmem = *tmem_ptr;
  in_turn();  // the setup has run beside the last blocks of the kernel before

  // a pair's epilogue warps take the registers that its control warps do not need
  if (warp >= 4) {
    // ---- epilogue
    if (CTAS == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpilogueRegs));
    const int quad = warp & 3, group = (warp - 4) >> 2;
    char* staging = staging_base + (warp - 4) * kStagingBytes;
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16) + group * 64;
    int acc = 0;
    uint32_t acc_phase = 0;
    // the accumulator has been read: the next product may write over it
    auto release = [&] {
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive_cluster(in_block(acc_empty(acc), 0));
      if ((acc ^= 1) == 0) acc_phase ^= 1;
    };
    auto ready = [&] {  // the warp stays whole
      const bool ok = __all_sync(0xffffffffu, wait(acc_full(acc), acc_phase));
      tmem_fence_after();
      return ok;
    };
    bool ok = true;
    for (uint32_t u = first_unit; u < units && ok; u += unit_step) {
      const Tile t = tile_of<CTAS>(P, u);
      const int64_t row0 = t.m0 + rank * kRowsPerBlock + quad * 32;
      const int col0 = t.n0 + group * 64;
      const bool inside = row0 < P.m && col0 < P.n;
      if constexpr (Epilogue::kFold) {
        f2 c[2][16];
        for (int k0 = 0; k0 < t.slabs; k0 += kFoldSlabs) {
          if (!(ok = ready())) break;
          const uint32_t at = lanes + acc * kTileN;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float v[16];
            tmem_load16(at + 16 * q, v);
            tmem_wait_load();
            tmem_hold16(v);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              f2& s = c[q / 2][q % 2 * 8 + i];
              s = k0 ? add2(s, pair(v[2 * i], v[2 * i + 1])) : pair(v[2 * i], v[2 * i + 1]);
            }
          }
          release();
        }
        if (!ok) break;
#pragma unroll
        for (int q = 0; q < 2; ++q)
          if (inside && col0 + 32 * q < P.n) E.run(c[q], row0, P.m, col0 + 32 * q, P.n, t.split, staging);
      } else {
        typename Epilogue::Ahead ahead;
        if (inside) E.prepare(ahead, row0, P.m, col0, P.n, staging);
        if (!(ok = ready())) break;
        const uint32_t at = lanes + acc * kTileN;
        auto load = [&](int half, f2(&z)[16]) {
          float v[32];
          tmem_load32(at + 32 * half, v);
          tmem_wait_load();
          tmem_hold32(v);
#pragma unroll
          for (int i = 0; i < 16; ++i) z[i] = pair(v[2 * i], v[2 * i + 1]);
        };
        if (inside) E.run(ahead, load, release, consts, row0, P.m, col0, P.n, staging);
        else release();
      }
    }
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // the stores have landed
  } else {
    if (CTAS == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kControlRegs));
    if (warp == 0 && lane == 0) {
      // ---- copies
      int st = 0;
      uint32_t phase = 0;
      int64_t issued = 0;
      bool ok = true;
      Tile next = tile_of<CTAS>(P, first_unit);
      for (uint32_t u = first_unit; u < units && ok; u += unit_step) {
        const Tile t = next;
        const int32_t ma = (int32_t)(t.m0 + rank * kRowsPerBlock), nb = t.n0 + (int)rank * kRowsPerBlock;
        for (int k = 0; k < t.slabs; ++k) {
          // the next tile's divisions under this tile's copies: at its start they would leave the ring empty
          if (k == 1 || t.slabs == 1) next = tile_of<CTAS>(P, u + unit_step);
          if (!wait(empty(st), phase ^ 1)) {
            ok = false;
            break;
          }
          if (rank == 0) bar_expect(full(st), CTAS * kStageBytes + P.stall_tx);
          const uint32_t bar = CTAS == 2 ? in_block(full(st), 0) : full(st);
          const uint32_t da = smem_addr(smem + st * kStageBytes), db = da + kOperandBytes;
          const int32_t kk = (t.first + k) * kSlabK;
          if (A_MN) {
            copy_box<CTAS>(da, &P.a, ma, kk, bar);
            copy_box<CTAS>(da + kOperandBytes / 2, &P.a, ma + 64, kk, bar);
          } else {
            copy_box<CTAS>(da, &P.a, kk, ma, bar);
          }
          if (B_MN) {
            copy_box<CTAS>(db, &P.b, nb, kk, bar);
            copy_box<CTAS>(db + kOperandBytes / 2, &P.b, nb + 64, kk, bar);
          } else {
            copy_box<CTAS>(db, &P.b, kk, nb, bar);
          }
          ++issued;
          if (++st == kStages) st = 0, phase ^= 1;
        }
      }
      if (!ok && rank == 0) {
        // gave up: the copies in flight land before the block leaves (a limited wait for each stage's)
        for (int64_t q = issued > kStages ? issued - kStages : 0; q < issued; ++q) {
          const long long t0 = clock64();
          while (!bar_try(full((int)(q % kStages)), (uint32_t)(q / kStages) & 1) && clock64() - t0 < 20000000ll) {
          }
        }
      }
    } else if (warp == 1 && lane == 0 && rank == 0) {
      // ---- products
      const uint32_t desc_a = operand_desc<A_MN>(smem_addr(smem)), desc_b = operand_desc<B_MN>(smem_addr(smem) + kOperandBytes);
      int st = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (uint32_t u = first_unit; u < units && ok; u += unit_step) {
        // nothing but the number of slabs, and that without a division where it is always the same: the tensor
        // cores run dry while this thread computes
        const int slabs = P.splits == 1 ? P.slabs : slabs_of(P, (int)(u % P.splits));
        for (int k0 = 0, k1; k0 < slabs && ok; k0 = k1) {
          k1 = Epilogue::kFold && slabs - k0 > kFoldSlabs ? k0 + kFoldSlabs : slabs;
          if (!(ok = wait(acc_empty(acc), acc_phase ^ 1))) break;
          tmem_fence_after();
          const uint32_t d = tmem + acc * kTileN;
          for (int k = k0; k < k1; ++k) {
            if (!(ok = wait(full(st), phase))) break;
            mma_slab<CTAS, A_MN, B_MN>(d, desc_a + st * (kStageBytes >> 4), desc_b + st * (kStageBytes >> 4), P.idesc, k > k0);
            mma_commit<CTAS>(empty(st));
            if (++st == kStages) st = 0, phase ^= 1;
          }
          if (!ok) break;
          mma_commit<CTAS>(acc_full(acc));
          if ((acc ^= 1) == 0) acc_phase ^= 1;
        }
      }
      // the tensor cores are done with shared and tensor memory before the block frees them
      mma_commit<CTAS>(drained);
      const long long t0 = clock64();
      while (!bar_try(drained, 0) && clock64() - t0 < 2000000000ll) {
      }
    }
  }
  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  if (CTAS == 2) cluster_sync();  // neither block leaves while the other may still reach into it
  tmem_fence_after();
  if (warp == 1) tmem_free<CTAS>(tmem, kTmemCols);
}

// ------------------------------------------------------------------------------------------------
// host side

// A row-major matrix of rows x cols 16-bit values, copied in boxes of 64 columns by box_rows rows.  The
// base lies on 16 bytes and ld is a multiple of 8.
cudaError_t make_map(CUtensorMap* map, int32_t dtype, const void* p, int64_t rows, int64_t cols, int64_t ld, int box_rows);
// An output matrix of elements of `size` bytes (1: codes), stored in boxes of 32 rows of 64 bytes (codes: 32).
cudaError_t make_output_map(CUtensorMap* map, int size, const void* p, int64_t rows, int64_t cols, int64_t ld);
template <typename T>
cudaError_t make_output(Output<T>* out, T* p, int64_t rows, int64_t cols, int64_t ld) {
  *out = Output<T>{};
  out->p = p;
  out->ld = ld;
  if (!p || !aligned(p, 16) || ld * (int64_t)sizeof(T) % 16 != 0) return cudaSuccess;
  out->by_tma = true;
  return make_output_map(&out->map, (int)sizeof(T), p, rows, cols, ld);
}
unsigned int* status_word();   // of the current device (NULL: a CUDA error)
uint32_t stall_bytes();        // the test hook's

struct ProductShape {
  int64_t m;
  int64_t n, k;
};
struct ProductPlan {
  int ctas, splits, split_slabs;
};
ProductPlan plan_product(const ProductShape& s, int sms);

struct Operand {
  const void* p;
  int64_t ld;
};

template <int CTAS, bool A_MN, bool B_MN, class Epilogue>
cudaError_t launch_product(const ProductArgs& P, const Epilogue& E, int sms, cudaStream_t s) {
  auto* kernel = k_product<CTAS, A_MN, B_MN, Epilogue>;
  static std::atomic<uint64_t> ready{0};  // devices on which this kernel may use its shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (!(ready.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kProductSmem<CTAS>);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  const int64_t units = P.units, most = sms / CTAS;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((units < most ? units : most) * CTAS));
  cfg.blockDim = dim3(kProductThreads<CTAS>);
  cfg.dynamicSmemBytes = kProductSmem<CTAS>;
  cfg.stream = s;
  cudaLaunchAttribute attr[2]{};
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CTAS;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, P, E);
}

// C = A B^T by `plan`, through epilogue E.  A: m x k (or k x m with A_MN), B: n x k (or k x n with B_MN).
template <int CTAS, bool A_MN, bool B_MN, class Epilogue>
cudaError_t run_product_by(int32_t dtype, const Operand& a, const Operand& b, const ProductShape& s, const ProductPlan& plan, const Epilogue& E,
                           cudaStream_t stream) {
  ProductArgs P{};
  cudaError_t e = make_map(&P.a, dtype, a.p, A_MN ? s.k : s.m, A_MN ? s.m : s.k, a.ld, A_MN ? 64 : 128);
  if (e == cudaSuccess) e = make_map(&P.b, dtype, b.p, B_MN ? s.k : s.n, B_MN ? s.n : s.k, b.ld, B_MN ? 64 : 128);
  if (e != cudaSuccess) return e;
  P.m = s.m;
  P.n = (int32_t)s.n;
  P.slabs = (int32_t)ceil_div(s.k, kSlabK);
  P.tiles_m = (int32_t)ceil_div(s.m, kRowsPerBlock * plan.ctas);
  P.tiles_n = (int32_t)ceil_div(s.n, kRowsPerBlock * plan.ctas);
  P.splits = plan.splits;
  P.split_slabs = plan.split_slabs;
  const int64_t units = (int64_t)P.tiles_m * P.tiles_n * P.splits;
  if (units >= (int64_t)1 << 31) return cudaErrorNotSupported;
  P.units = (uint32_t)units;
  const uint32_t per = (uint32_t)kGroupTiles * (uint32_t)P.tiles_n;  // at least 8
  P.group_shift = 32 - (uint32_t)__builtin_clz(per - 1);
  P.group_mul = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << P.group_shift) - per)) / per + 1);
  const uint32_t type = dtype == ONEBIT_F16 ? 0u : 1u;  // both operands have the same
  P.idesc = 1u << 4 | type << 7 | type << 10 | (uint32_t)A_MN << 15 | (uint32_t)B_MN << 16 |
            (uint32_t)(kRowsPerBlock * plan.ctas / 8) << 17 | (uint32_t)(kRowsPerBlock * plan.ctas / 16) << 24;
  P.stall_tx = stall_bytes();
  P.status = status_word();
  if (!P.status) return cudaErrorUnknown;
  return launch_product<CTAS, A_MN, B_MN>(P, E, sm_count(), stream);
}
template <bool A_MN, bool B_MN, class Epilogue>
cudaError_t run_product(int32_t dtype, const Operand& a, const Operand& b, const ProductShape& s, const ProductPlan& plan, const Epilogue& E,
                        cudaStream_t stream) {
  return plan.ctas == 2 ? run_product_by<2, A_MN, B_MN>(dtype, a, b, s, plan, E, stream)
                        : run_product_by<1, A_MN, B_MN>(dtype, a, b, s, plan, E, stream);
}

}  // namespace layers
}  // namespace onebit
