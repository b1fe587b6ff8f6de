// gated_forward.cu -- the gated linear layer's forward pass: both projections in one matrix product, activation,
// gating and what is kept.  See include/onebit_layers.h for the formulas.
#include "gated_common.cuh"

namespace onebit {
namespace layers {
namespace {

// What the product's epilogue does for one call.
template <typename T>
struct GatedOut {
  const float* bias;
  T* h;
  int64_t ldh;
  T* z;
  int64_t ldz;
  int8_t *gate_codes, *up_codes;
  float *gate_scales, *up_scales;
  int blocks, act;
};

// The epilogue over the sums z (partial ones of a cut contraction), one warp per 64 columns of a row of h.
template <typename T>
__global__ void __launch_bounds__(256) k_finish_gated(Partials c, int64_t rows, int n, const GatedOut<T> o) {
  in_turn();
  const int lane = threadIdx.x & 31;
  const int64_t units = rows * o.blocks, step = (int64_t)gridDim.x * 8;
  for (int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); i < units; i += step) {
    const int64_t r = i / o.blocks;
    const int c0 = (int)(i - r * o.blocks) * kBlock + lane;
    float g[2], u[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int col = c0 + 32 * q;
      g[q] = u[q] = 0.0f;
      if (col < n) {
        g[q] = c.at(r, col) + (o.bias ? o.bias[col] : 0.0f);
        u[q] = c.at(r, n + col) + (o.bias ? o.bias[n + col] : 0.0f);
        o.h[r * o.ldh + col] = from_f<T>(gate_both(o.act, g[q]).x * u[q]);
        if (o.z) o.z[r * o.ldz + col] = from_f<T>(g[q]), o.z[r * o.ldz + n + col] = from_f<T>(u[q]);
      }
    }
    if (o.gate_codes) {
      const BlockScale sg = block_scale(warp_max_nan(max_nan(fabsf(g[0]), fabsf(g[1])))), su = block_scale(warp_max_nan(max_nan(fabsf(u[0]), fabsf(u[1]))));
#pragma unroll
      for (int q = 0; q < 2; ++q)
        if (c0 + 32 * q < n) {
          o.gate_codes[r * n + c0 + 32 * q] = (int8_t)code_of(g[q], sg.inv);
          o.up_codes[r * n + c0 + 32 * q] = (int8_t)code_of(u[q], su.inv);
        }
      if (lane == 0) o.gate_scales[i] = sg.scale, o.up_scales[i] = su.scale;
    }
  }
}

// Takes the workspace; with `run`, enqueues the work too.
template <typename T>
cudaError_t forward(const onebit_gated_linear_t& a, Space& ws, cudaStream_t s, bool run) {
  const ProductShape shape{a.rows, 2 * a.inner, a.in};
  ProductPlan plan = plan_product(shape, sm_count());
  Readable copies;
  const Operand x = copies.take(ws, a.x, a.ldx, a.rows, a.in), w = copies.take(ws, a.w, a.ldw, 2 * a.inner, a.in);
  const Partials part = take_sums(ws, plan, a.rows, 2 * a.inner);
  if (!run) return cudaSuccess;
  cudaError_t err = copies.run(s);
  if (err != cudaSuccess) return err;
  PlainEpilogue<float> to{};
  err = to_partials(&to, part, 2 * a.inner);
  if (err == cudaSuccess) err = run_product<false, false>(a.dtype, x, w, shape, plan, to, s);
  if (err != cudaSuccess) return err;
  const int64_t blocks = ceil_div(a.inner, kBlock);
  const GatedOut<T> o{a.bias, static_cast<T*>(a.h), a.ldh, static_cast<T*>(a.z), a.ldz, a.gate_codes, a.up_codes, a.gate_scales, a.up_scales,
                      (int)blocks, a.activation};
  return launch_after(k_finish_gated<T>, flat_grid(a.rows * blocks * 32, 256), 256, s, part, a.rows, (int)a.inner, o);
}
cudaError_t forward(const onebit_gated_linear_t& a, Space& ws, cudaStream_t s, bool run) {
  return a.dtype == ONEBIT_F16 ? forward<__half>(a, ws, s, run) : forward<__nv_bfloat16>(a, ws, s, run);
}

onebit_status_t forward_ok(const onebit_gated_linear_t* a) {
  if (!a) return fail(ONEBIT_ERR_INVALID_ARG, "the arguments are NULL");
  onebit_status_t st = gated_shape_ok(a->rows, a->in, a->inner, a->dtype, a->activation);
  if (st != ONEBIT_OK) return st;
  if (a->ldx < a->in || a->ldw < a->in || a->ldh < a->inner || (a->z && a->ldz < 2 * a->inner))
    return fail(ONEBIT_ERR_INVALID_ARG, "a row stride below the columns");
  if (!checkpoints_whole(a->gate_codes, a->gate_scales, a->up_codes, a->up_scales))
    return fail(ONEBIT_ERR_INVALID_ARG, "checkpoints need the codes and scales of both halves");
  if (a->z && a->gate_codes) return fail(ONEBIT_ERR_INVALID_ARG, "what is kept is z or its checkpoints, not both");
  if (a->rows > 0 && (!a->x || !a->w || !a->h)) return fail(ONEBIT_ERR_INVALID_ARG, "a NULL buffer");
  if (!aligned(a->x, 2) || !aligned(a->w, 2) || !aligned(a->h, 2) || !aligned(a->z, 2) || !aligned(a->bias, 4) || !aligned(a->gate_scales, 4) ||
      !aligned(a->up_scales, 4))
    return fail(ONEBIT_ERR_INVALID_ARG, "a buffer is not aligned to its type");
  return ONEBIT_OK;
}

}  // namespace
}  // namespace layers
}  // namespace onebit

using namespace onebit::layers;

extern "C" onebit_status_t onebit_gated_linear_forward_workspace(const onebit_gated_linear_t* a, size_t* bytes) {
  onebit_status_t st = forward_ok(a);
  if (st != ONEBIT_OK) return st;
  if (!bytes) return fail(ONEBIT_ERR_INVALID_ARG, "bytes is NULL");
  Space ws{nullptr};
  if (a->rows > 0) forward(*a, ws, nullptr, false);
  *bytes = (size_t)ws.used;
  return ONEBIT_OK;
}

extern "C" onebit_status_t onebit_gated_linear_forward(const onebit_gated_linear_t* a, void* workspace, size_t workspace_bytes,
                                                       onebit_stream_t stream) {
  size_t need = 0;
  onebit_status_t st = onebit_gated_linear_forward_workspace(a, &need);
  if (st != ONEBIT_OK || a->rows == 0) return st;
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256)))
    return fail(ONEBIT_ERR_WORKSPACE, "the workspace is too small or not 256-byte aligned");
  const int64_t codes = a->rows * a->inner, scales = a->rows * ceil_div(a->inner, kBlock) * 4;
  if (!disjoint({matrix(a->x, a->rows, a->ldx, a->in, 2), matrix(a->w, 2 * a->inner, a->ldw, a->in, 2), span_of(a->bias, 2 * a->inner * 4)},
                {matrix(a->h, a->rows, a->ldh, a->inner, 2), matrix(a->z, a->rows, a->ldz, 2 * a->inner, 2), span_of(a->gate_codes, codes),
                 span_of(a->gate_scales, scales), span_of(a->up_codes, codes), span_of(a->up_scales, scales), span_of(workspace, (int64_t)need)}))
    return fail(ONEBIT_ERR_INVALID_ARG, "an output overlaps another buffer");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  Space ws{static_cast<char*>(workspace)};
  const cudaError_t e = forward(*a, ws, s, true);
  return e == cudaSuccess ? ONEBIT_OK : cuda_fail(e, "onebit_gated_linear_forward");
}
