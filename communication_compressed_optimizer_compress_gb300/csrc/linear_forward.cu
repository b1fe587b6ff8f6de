// linear_forward.cu -- the linear layer's forward pass: matrix product with bias, activation, residual
// and an 8-bit checkpoint in its epilogue.  See include/onebit_layers.h for the formulas.
#include "few_rows.cuh"

namespace onebit {
namespace layers {
namespace {

// The epilogue over the partial sums of a cut contraction, one warp per 64 columns of a row.
template <typename T>
__global__ void __launch_bounds__(256) k_finish_forward(Partials c, int64_t rows, int cols, const __grid_constant__ ForwardEpilogue<T, kAny, kAny, kAny> e) {
  in_turn();
  const int lane = threadIdx.x & 31;
  const int64_t units = rows * e.blocks, step = (int64_t)gridDim.x * 8;
  for (int64_t u = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); u < units; u += step) {
    const int64_t r = u / e.blocks;
    const int c0 = (int)(u - r * e.blocks) * kBlock + lane;
    float z[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int col = c0 + 32 * q;
      z[q] = 0.0f;
      if (col < cols) {
        z[q] = c.at(r, col) + (e.bias ? e.bias[col] : 0.0f);
        float v = act_value(e.act, z[q]);
        if (e.residual.p) v += to_f(e.residual.p[r * e.residual.ld + col]);
        e.y.p[r * e.y.ld + col] = from_f<T>(v);
      }
    }
    if (e.scales) {
      const BlockScale s = block_scale(warp_max_nan(max_nan(fabsf(z[0]), fabsf(z[1]))));
#pragma unroll
      for (int q = 0; q < 2; ++q)
        if (c0 + 32 * q < cols) e.codes.p[r * cols + c0 + 32 * q] = (int8_t)code_of(z[q], s.inv);
      if (lane == 0) e.scales[u] = s.scale;
    }
  }
}

// Takes the workspace; with `run`, enqueues the work too.
template <typename T>
cudaError_t forward(const onebit_linear_t& a, Space& ws, cudaStream_t s, bool run) {
  if (few_rows(a)) return run ? run_few_rows<T>(a, s) : cudaSuccess;
  const ProductShape shape{a.rows, a.out, a.in};
  const ProductPlan plan = plan_product(shape, sm_count());
  Readable copies;
  const Operand x = copies.take(ws, a.x, a.ldx, a.rows, a.in), w = copies.take(ws, a.w, a.ldw, a.out, a.in);
  const Partials part = take_partials(ws, plan, a.rows, a.out);
  if (!run) return cudaSuccess;
  cudaError_t err = copies.run(s);
  if (err != cudaSuccess) return err;
  ForwardEpilogue<T, kAny, kAny, kAny> e{};
  e.bias = a.bias;
  e.residual = make_input<T>(a.residual, a.ldr);
  e.scales = a.scales;
  e.blocks = (int)ceil_div(a.out, kBlock);
  e.act = a.activation;
  err = make_output(&e.y, static_cast<T*>(a.y), a.rows, a.out, a.ldy);
  if (err == cudaSuccess) err = make_output(&e.codes, a.codes, a.rows, a.out, a.out);
  if (err != cudaSuccess) return err;
  if (plan.splits == 1 && plan.ctas == 1) return run_product_by<1, false, false>(a.dtype, x, w, shape, plan, e, s);
  if (plan.splits == 1) {
    using std::integral_constant;
    using Any = integral_constant<int, kAny>;
    auto go = [&](auto act, auto ck, auto res) {
      ForwardEpilogue<T, decltype(act)::value, decltype(ck)::value, decltype(res)::value> f{};
      f.bias = e.bias, f.residual = e.residual, f.y = e.y, f.codes = e.codes, f.scales = e.scales, f.blocks = e.blocks, f.act = e.act;
      return run_product_by<2, false, false>(a.dtype, x, w, shape, plan, f, s);
    };
    using No = integral_constant<int, 0>;
    using Yes = integral_constant<int, 1>;
    using None = integral_constant<int, ONEBIT_ACT_NONE>;
    if (a.residual) return a.activation == ONEBIT_ACT_NONE && !a.codes ? go(None{}, No{}, Yes{}) : go(Any{}, Any{}, Any{});
    auto by_act = [&](auto ck) {
      switch (a.activation) {
        case ONEBIT_ACT_RELU: return go(integral_constant<int, ONEBIT_ACT_RELU>{}, ck, No{});
        case ONEBIT_ACT_GELU: return go(integral_constant<int, ONEBIT_ACT_GELU>{}, ck, No{});
        case ONEBIT_ACT_GELU_TANH: return go(integral_constant<int, ONEBIT_ACT_GELU_TANH>{}, ck, No{});
        default: return go(None{}, ck, No{});
      }
    };
    return a.codes ? by_act(Yes{}) : by_act(No{});
  }
  PlainEpilogue<float> to{};
  err = to_partials(&to, part, a.out);
  if (err == cudaSuccess) err = run_product<false, false>(a.dtype, x, w, shape, plan, to, s);
  if (err != cudaSuccess) return err;
  return launch_after(k_finish_forward<T>, flat_grid(a.rows * e.blocks * 32, 256), 256, s, part, a.rows, (int)a.out, e);
}
cudaError_t forward(const onebit_linear_t& a, Space& ws, cudaStream_t s, bool run) {
  return a.dtype == ONEBIT_F16 ? forward<__half>(a, ws, s, run) : forward<__nv_bfloat16>(a, ws, s, run);
}

onebit_status_t forward_ok(const onebit_linear_t* a) {
  if (!a) return fail(ONEBIT_ERR_INVALID_ARG, "the arguments are NULL");
  onebit_status_t st = linear_shape_ok(a->rows, a->in, a->out, a->dtype, a->activation);
  if (st != ONEBIT_OK) return st;
  if (a->ldx < a->in || a->ldw < a->in || a->ldy < a->out || (a->residual && a->ldr < a->out))
    return fail(ONEBIT_ERR_INVALID_ARG, "a row stride below the columns");
  if (!a->codes != !a->scales) return fail(ONEBIT_ERR_INVALID_ARG, "a checkpoint needs codes and scales");
  if (a->rows > 0 && (!a->x || !a->w || !a->y)) return fail(ONEBIT_ERR_INVALID_ARG, "a NULL buffer");
  if (!aligned(a->x, 2) || !aligned(a->w, 2) || !aligned(a->y, 2) || !aligned(a->residual, 2) || !aligned(a->bias, 4) ||
      !aligned(a->scales, 4))
    return fail(ONEBIT_ERR_INVALID_ARG, "a buffer is not aligned to its type");
  return ONEBIT_OK;
}

}  // namespace
}  // namespace layers
}  // namespace onebit

using namespace onebit::layers;

extern "C" onebit_status_t onebit_linear_forward_workspace(const onebit_linear_t* a, size_t* bytes) {
  onebit_status_t st = forward_ok(a);
  if (st != ONEBIT_OK) return st;
  if (!bytes) return fail(ONEBIT_ERR_INVALID_ARG, "bytes is NULL");
  Space ws{nullptr};
  if (a->rows > 0) forward(*a, ws, nullptr, false);
  *bytes = (size_t)ws.used;
  return ONEBIT_OK;
}

extern "C" onebit_status_t onebit_linear_forward(const onebit_linear_t* a, void* workspace, size_t workspace_bytes,
                                                 onebit_stream_t stream) {
  size_t need = 0;
  onebit_status_t st = onebit_linear_forward_workspace(a, &need);
  if (st != ONEBIT_OK || a->rows == 0) return st;
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256)))
    return fail(ONEBIT_ERR_WORKSPACE, "the workspace is too small or not 256-byte aligned");
  const int64_t blocks = ceil_div(a->out, kBlock);
  if (!disjoint({matrix(a->x, a->rows, a->ldx, a->in, 2), matrix(a->w, a->out, a->ldw, a->in, 2),
                 span_of(a->bias, a->out * 4), matrix(a->residual, a->rows, a->ldr, a->out, 2)},
                {matrix(a->y, a->rows, a->ldy, a->out, 2), span_of(a->codes, a->rows * a->out),
                 span_of(a->scales, a->rows * blocks * 4), span_of(workspace, (int64_t)need)}))
    return fail(ONEBIT_ERR_INVALID_ARG, "an output overlaps another buffer");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  Space ws{static_cast<char*>(workspace)};
  const cudaError_t e = forward(*a, ws, s, true);
  return e == cudaSuccess ? ONEBIT_OK : cuda_fail(e, "onebit_linear_forward");
}
