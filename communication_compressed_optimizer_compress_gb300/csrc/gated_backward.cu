// gated_backward.cu -- the backward pass through the product behind a gated linear layer, to the gate and up values
// before the gating, with dw and db.  See include/onebit_layers.h for the formulas.
#include "gated_common.cuh"

namespace onebit {
namespace layers {
namespace {

// g and u as the backward pass has them.
template <typename T>
struct KeptPair {
  Kept<T> gate, up;
};

// dz from the sums dh (partial ones of a cut contraction), and h = act(g) u, a warp for 128 columns of a row, single elements side
// by side, which serves rows of any alignment.  Without dz: h alone.  Bound by latency at the sizes that come here (333 x 1030: 3 us of the
// 13 that dz takes); a large dz from sums moves them through DRAM (16384 x 4090: 531 us, 432 in the epilogue).
template <typename T>
__global__ void __launch_bounds__(256) k_finish_dz(Partials c, int64_t rows, int n, KeptPair<T> kept, int act, T* __restrict__ dz, int64_t lddz,
                                                   T* __restrict__ h, int64_t ldh) {
  in_turn();
  const int lane = threadIdx.x & 31;
  const int64_t per = (n + 127) / 128, units = rows * per, step = (int64_t)gridDim.x * 8;
  for (int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); i < units; i += step) {
    const int64_t r = i / per;
    const int c0 = (int)(i - r * per) * 128 + lane;
    float d[4], g[4], u[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int col = c0 + 32 * q;
      d[q] = g[q] = u[q] = 0.0f;
      if (col < n) {
        g[q] = kept.gate.at(r, col), u[q] = kept.up.at(r, col);
        if (dz) d[q] = c.at(r, col);
      }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int col = c0 + 32 * q;
      if (col >= n) break;
      const float2 p = gate_both(act, g[q]);
      if (h) h[r * ldh + col] = from_f<T>(p.x * u[q]);
      if (dz) dz[r * lddz + col] = from_f<T>(d[q] * u[q] * p.y), dz[r * lddz + n + col] = from_f<T>(d[q] * p.x);
    }
  }
}

// Takes the workspace; with `run`, enqueues the work too.
template <typename T>
cudaError_t backward(const onebit_gated_linear_grad_t& a, Space& ws, cudaStream_t s, bool run) {
  const int blocks = (int)ceil_div(a.inner, kBlock), n = (int)a.inner;
  const T* z = static_cast<const T*>(a.z);
  const KeptPair<T> kept{{z, a.ldz, a.gate_codes, a.gate_scales, n, blocks}, {z ? z + n : nullptr, a.ldz, a.up_codes, a.up_scales, n, blocks}};
  const int64_t ldh = pad8(a.inner);
  T* h = a.dw ? ws.take<T>(a.rows * ldh) : nullptr;  // rounded as the forward pass rounded what it multiplied w with
  Readable copies;
  Operand dy{a.dy, a.lddy}, w{};
  if (a.dz) dy = copies.take(ws, a.dy, a.lddy, a.rows, a.out), w = copies.take(ws, a.w, a.ldw, a.out, a.inner);
  cudaError_t err = run ? copies.run(s) : cudaSuccess;
  if (err != cudaSuccess) return err;
  Partials part{};
  bool done = false;  // dz and h, in the epilogue
  if (a.dz) {
    const ProductShape shape{a.rows, a.inner, a.out};
    const ProductPlan plan = plan_product(shape, sm_count());
    // Single blocks that cannot store dz by TMA leave it to the kernel over the sums: their few warps write it element by element
    // (333 x 1030 x 520: 19.8 us from values in the epilogue, 13.0 that way; pairs have more work each: 16384 x 4090 x 1024 432 and 531).
    const bool whole = aligned(a.dz, 16) && a.lddz % 8 == 0 && a.inner % 8 == 0, fused = plan.splits == 1 && (whole || plan.ctas == 2);
    if (!fused) part = take_sums(ws, plan, a.rows, a.inner);
    if (run && fused) {
      auto go = [&](auto ctas, auto act, auto what) {
        GatedGradEpilogue<T, decltype(act)::value, decltype(what)::value> e{};
        e.gate = make_input<T>(kept.gate.x, a.ldz), e.up = make_input<T>(kept.up.x, a.ldz);
        e.gate_codes = a.gate_codes, e.up_codes = a.up_codes, e.gate_scales = a.gate_scales, e.up_scales = a.up_scales;
        e.blocks = blocks, e.act = a.activation, e.kept = a.z ? kKeptValue : kKeptCodes;
        e.code_bytes = aligned(a.gate_codes, 16) && aligned(a.up_codes, 16) && n % 16 == 0 ? 16 : aligned(a.gate_codes, 8) && aligned(a.up_codes, 8) && n % 8 == 0 ? 8 : 1;
        T* dz = static_cast<T*>(a.dz);
        cudaError_t r = make_output(&e.dgate, dz, a.rows, a.inner, a.lddz);
        if (r == cudaSuccess) r = make_output(&e.dup, dz + n, a.rows, a.inner, a.lddz);
        if (r == cudaSuccess) r = make_output(&e.h, h, a.rows, a.inner, ldh, true);
        return r == cudaSuccess ? run_product_by<decltype(ctas)::value, false, true>(a.dtype, dy, w, shape, plan, e, s) : r;
      };
      using std::integral_constant;
      using Any = integral_constant<int, kAny>;
      auto by_act = [&](auto what) {
        integral_constant<int, 2> two;
        switch (a.activation) {
          case ONEBIT_ACT_GELU: return go(two, integral_constant<int, ONEBIT_ACT_GELU>{}, what);
          case ONEBIT_ACT_GELU_TANH: return go(two, integral_constant<int, ONEBIT_ACT_GELU_TANH>{}, what);
          case ONEBIT_ACT_SILU: return go(two, integral_constant<int, ONEBIT_ACT_SILU>{}, what);
          case ONEBIT_ACT_RELU: return go(two, integral_constant<int, ONEBIT_ACT_RELU>{}, what);
          default: return go(two, integral_constant<int, ONEBIT_ACT_NONE>{}, what);
        }
      };
      err = plan.ctas == 1 ? go(integral_constant<int, 1>{}, Any{}, Any{})
            : a.z          ? by_act(integral_constant<int, kKeptValue>{}) : by_act(integral_constant<int, kKeptCodes>{});
      if (err != cudaSuccess) return err;
      done = true;
    } else if (run) {
      PlainEpilogue<float> to{};
      err = to_partials(&to, part, a.inner);
      if (err == cudaSuccess) err = run_product<false, true>(a.dtype, dy, w, shape, plan, to, s);
      if (err != cudaSuccess) return err;
    }
  }
  if (run && !done && (a.dz || h)) {
    err = launch_after(k_finish_dz<T>, flat_grid(a.rows * ceil_div(a.inner, 128) * 32, 256), 256, s, part, a.rows, n, kept, a.activation, static_cast<T*>(a.dz),
                       a.lddz, h, ldh);
    if (err != cudaSuccess) return err;
  }
  if (!a.dw && !a.db) return cudaSuccess;
  onebit_linear_grad_t b{};
  b.dy = dy.p, b.lddy = dy.ld, b.x = h, b.ldx = ldh, b.dw = a.dw, b.db = a.db;
  b.rows = a.rows, b.in = a.inner, b.out = a.out, b.dtype = a.dtype, b.grad_dtype = a.grad_dtype;
  return linear_backward(b, ws, s, run, dy.p != a.dy);
}
cudaError_t backward(const onebit_gated_linear_grad_t& a, Space& ws, cudaStream_t s, bool run) {
  return a.dtype == ONEBIT_F16 ? backward<__half>(a, ws, s, run) : backward<__nv_bfloat16>(a, ws, s, run);
}

onebit_status_t backward_ok(const onebit_gated_linear_grad_t* a) {
  if (!a) return fail(ONEBIT_ERR_INVALID_ARG, "the arguments are NULL");
  onebit_status_t st = gated_shape_ok(a->rows, a->out, a->inner, a->dtype, a->activation);
  if (st != ONEBIT_OK) return st;
  if (!dtype_ok(a->grad_dtype)) return fail(ONEBIT_ERR_INVALID_ARG, "grad_dtype is not one of f32, f16, bf16");
  if (!checkpoints_whole(a->gate_codes, a->gate_scales, a->up_codes, a->up_scales))
    return fail(ONEBIT_ERR_INVALID_ARG, "checkpoints need the codes and scales of both halves");
  if (a->z && a->gate_codes) return fail(ONEBIT_ERR_INVALID_ARG, "what was kept is z or its checkpoints, not both");
  if (a->lddy < a->out || (a->z && a->ldz < 2 * a->inner) || (a->dz && (a->ldw < a->inner || a->lddz < 2 * a->inner)))
    return fail(ONEBIT_ERR_INVALID_ARG, "a row stride below the columns");
  if (a->rows > 0) {
    if ((a->dz || a->dw || a->db) && !a->dy) return fail(ONEBIT_ERR_INVALID_ARG, "a NULL buffer");
    if (a->dz && !a->w) return fail(ONEBIT_ERR_INVALID_ARG, "dz needs the weight");
    if ((a->dz || a->dw) && !a->z && !a->gate_codes) return fail(ONEBIT_ERR_INVALID_ARG, "dz and dw need z or its checkpoints");
  }
  const uintptr_t g = (uintptr_t)dtype_size(a->grad_dtype);
  if (!aligned(a->dy, 2) || !aligned(a->z, 2) || !aligned(a->w, 2) || !aligned(a->dz, 2) || !aligned(a->gate_scales, 4) ||
      !aligned(a->up_scales, 4) || !aligned(a->dw, g) || !aligned(a->db, g))
    return fail(ONEBIT_ERR_INVALID_ARG, "a buffer is not aligned to its type");
  return ONEBIT_OK;
}

}  // namespace
}  // namespace layers
}  // namespace onebit

using namespace onebit::layers;

extern "C" onebit_status_t onebit_gated_linear_backward_workspace(const onebit_gated_linear_grad_t* a, size_t* bytes) {
  onebit_status_t st = backward_ok(a);
  if (st != ONEBIT_OK) return st;
  if (!bytes) return fail(ONEBIT_ERR_INVALID_ARG, "bytes is NULL");
  Space ws{nullptr};
  if (a->rows > 0) backward(*a, ws, nullptr, false);
  *bytes = (size_t)ws.used;
  return ONEBIT_OK;
}

extern "C" onebit_status_t onebit_gated_linear_backward(const onebit_gated_linear_grad_t* a, void* workspace, size_t workspace_bytes,
                                                        onebit_stream_t stream) {
  size_t need = 0;
  onebit_status_t st = onebit_gated_linear_backward_workspace(a, &need);
  if (st != ONEBIT_OK) return st;
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256)))
    return fail(ONEBIT_ERR_WORKSPACE, "the workspace is too small or not 256-byte aligned");
  const int64_t codes = a->rows * a->inner, scales = a->rows * ceil_div(a->inner, kBlock) * 4, g = dtype_size(a->grad_dtype);
  if (!disjoint({matrix(a->dy, a->rows, a->lddy, a->out, 2), matrix(a->z, a->rows, a->ldz, 2 * a->inner, 2), span_of(a->gate_codes, codes),
                 span_of(a->gate_scales, scales), span_of(a->up_codes, codes), span_of(a->up_scales, scales),
                 matrix(a->w, a->out, a->ldw, a->inner, 2)},
                {matrix(a->dz, a->rows, a->lddz, 2 * a->inner, 2), span_of(a->dw, a->out * a->inner * g), span_of(a->db, a->out * g),
                 span_of(workspace, (int64_t)need)}))
    return fail(ONEBIT_ERR_INVALID_ARG, "an output overlaps another buffer");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (a->rows > 0) {
    Space ws{static_cast<char*>(workspace)};
    e = backward(*a, ws, s, true);
  } else {  // no tokens: the parameters' gradients are 0
    if (a->dw) e = cudaMemsetAsync(a->dw, 0, (size_t)(a->out * a->inner * g), s);
    if (a->db && e == cudaSuccess) e = cudaMemsetAsync(a->db, 0, (size_t)(a->out * g), s);
  }
  return e == cudaSuccess ? ONEBIT_OK : cuda_fail(e, "onebit_gated_linear_backward");
}
