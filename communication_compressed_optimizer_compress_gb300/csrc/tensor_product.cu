// tensor_product.cu -- host side of the tensor-core products: tensor maps, the plan, the status word.
#include "tensor_product.cuh"

#include <atomic>
#include <mutex>

namespace onebit {
namespace layers {

namespace {

constexpr int kMaxDevices = 64;
static __device__ unsigned int g_status;

std::mutex g_mu;
unsigned int* g_address[kMaxDevices] = {};
std::atomic<uint32_t> g_stall{0};

using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                            const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

Encode encoder() {
  static const Encode f = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<Encode>(p);
  }();
  return f;
}

}  // namespace

cudaError_t make_map(CUtensorMap* map, int32_t dtype, const void* p, int64_t rows, int64_t cols, int64_t ld, int box_rows) {
  const Encode encode = encoder();
  if (!encode) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  const cuuint32_t box[2] = {(cuuint32_t)kSlabK, (cuuint32_t)box_rows}, step[2] = {1, 1};
  const CUresult r = encode(map, dtype == ONEBIT_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                            const_cast<void*>(p), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t make_output_map(CUtensorMap* map, int size, const void* p, int64_t rows, int64_t cols, int64_t ld) {
  const Encode encode = encoder();
  if (!encode) return cudaErrorNotSupported;
  // bits only: the type decides nothing but its size
  const CUtensorMapDataType type = size == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : size == 2 ? CU_TENSOR_MAP_DATA_TYPE_UINT16 : CU_TENSOR_MAP_DATA_TYPE_UINT32;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)(ld * size)};
  const cuuint32_t box[2] = {size == 1 ? 32u : 64u / size, 32u}, step[2] = {1, 1};
  const CUresult r = encode(map, type, 2, const_cast<void*>(p), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            size == 1 ? CU_TENSOR_MAP_SWIZZLE_32B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

unsigned int* status_word() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  std::lock_guard<std::mutex> lock(g_mu);
  if (!g_address[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_status) != cudaSuccess) return nullptr;
    g_address[dev] = static_cast<unsigned int*>(p);
  }
  return g_address[dev];
}

uint32_t stall_bytes() { return g_stall.load(); }

// Which blocks and how many cuts of the contraction: the least of a model of the time, in SM clocks.
// A pair's 256x256 tile takes 512 clocks a slab, a single block's 128x128 tile about 330 (it reads
// twice the shared memory per product); a tile starts and ends in about 3000; cutting the contraction
// writes and reads fp32 partial tiles (about 3500 bytes a clock) and takes a second kernel.
ProductPlan plan_product(const ProductShape& s, int sms) {
  const int64_t slabs = ceil_div(s.k, kSlabK);
  ProductPlan best{2, 1, (int)slabs};
  double least = 1e300;
  for (int ctas = 1; ctas <= 2; ++ctas) {
    const int64_t tiles = ceil_div(s.m, kRowsPerBlock * ctas) * ceil_div(s.n, kRowsPerBlock * ctas), slots = sms / ctas > 0 ? sms / ctas : 1;
    for (int64_t want = 1; want <= 16 && (want == 1 || (slabs >= 4 * want && s.m * want < (int64_t)1 << 30)); ++want) {
      const int64_t per = ceil_div(slabs, want), splits = ceil_div(slabs, per);
      if (per > 1024 && want < 16) continue;  // one accumulator sums at most 65536 terms, where it can be helped
      const double waves = (double)ceil_div(tiles * splits, slots);
      double t = waves * ((double)per * (ctas == 2 ? 512.0 : 330.0)) + 3000.0;
      if (splits > 1) t += 5000.0 + (double)(s.m * s.n) * 8.0 * (double)splits / 3500.0;
      if (t < least) least = t, best = ProductPlan{ctas, (int)splits, (int)per};
    }
  }
  return best;
}

}  // namespace layers
}  // namespace onebit

using namespace onebit::layers;

extern "C" onebit_status_t onebit_layers_get_status(onebit_stream_t stream) {
  unsigned int* p = status_word();
  if (!p) return fail(ONEBIT_ERR_CUDA, "no status word on this device");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  unsigned int v = 0;
  cudaError_t e = cudaMemcpyAsync(&v, p, sizeof v, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return cuda_fail(e, "onebit_layers_get_status");
  return v & kStatusGaveUp ? fail(ONEBIT_ERR_CUDA, "a kernel gave up waiting for its copies or its cluster") : ONEBIT_OK;
}

extern "C" onebit_status_t onebit_layers_clear_status(onebit_stream_t stream) {
  unsigned int* p = status_word();
  if (!p) return fail(ONEBIT_ERR_CUDA, "no status word on this device");
  const cudaError_t e = cudaMemsetAsync(p, 0, sizeof(unsigned int), static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ONEBIT_OK : cuda_fail(e, "onebit_layers_clear_status");
}

extern "C" onebit_status_t onebit_layers_set_fault_injection(int32_t kind, int64_t value) {
  if (kind == ONEBIT_FAULT_NONE) {
    g_stall.store(0);
    return ONEBIT_OK;
  }
  if (kind != ONEBIT_FAULT_STALL_COPIES) return fail(ONEBIT_ERR_UNSUPPORTED, "only ONEBIT_FAULT_STALL_COPIES applies here");
  if (value < 1 || value > (1 << 19)) return fail(ONEBIT_ERR_INVALID_ARG, "stall bytes out of range");
  g_stall.store((uint32_t)value);
  return ONEBIT_OK;
}
