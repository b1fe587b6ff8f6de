// linear_backward.cu -- the linear layer's backward pass: dx through the derivative of the activation
// before the product, dw and db.  See include/onebit_layers.h for the formulas.
#include "linear_common.cuh"

namespace onebit {
namespace layers {
namespace {

// dx = (the product) * act'(v) [+ add] over the partial sums of a cut contraction, and h = act(v)
template <typename T>
__global__ void __launch_bounds__(256) k_finish_dx(Partials c, int64_t rows, int cols, Kept<T> v, int act, const T* __restrict__ add,
                                                   int64_t ldadd, T* __restrict__ dx, int64_t lddx, T* __restrict__ h, int64_t ldh) {
  in_turn();
  const int64_t per = c.ld / 4, total = rows * per;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / per;
    const int c0 = (int)(i - r * per) * 4;
    float d[4];
    c.at4(r, c0, d);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int col = c0 + q;
      if (col >= cols) break;
      if (act != ONEBIT_ACT_NONE || h) {
        const float2 p = act_both(act, v.at(r, col));
        d[q] *= p.y;
        if (h) h[r * ldh + col] = from_f<T>(p.x);
      }
      if (add) d[q] += to_f(add[r * ldadd + col]);
      dx[r * lddx + col] = from_f<T>(d[q]);
    }
  }
}

// h = act(v), rounded to the product's operand type, where dx is not computed beside it
template <typename T>
__global__ void __launch_bounds__(256) k_operand(Kept<T> v, int64_t rows, int cols, int act, T* __restrict__ h, int64_t ldh) {
  in_turn();
  const int64_t total = rows * cols;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / cols;
    const int col = (int)(i - r * cols);
    h[r * ldh + col] = from_f<T>(act_value(act, v.at(r, col)));
  }
}

// dw over the partial sums of a cut contraction, four columns a thread
template <typename G>
__global__ void __launch_bounds__(256) k_finish_dw(Partials c, int64_t rows, int cols, G* __restrict__ dw) {
  in_turn();
  const int64_t per = c.ld / 4, total = rows * per;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / per;
    const int c0 = (int)(i - r * per) * 4;
    float s[4];
    c.at4(r, c0, s);
    G* p = dw + r * cols + c0;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (c0 + q < cols) p[q] = from_f<G>(s[q]);
  }
}

// Column sums of dy over runs of kRun rows: a block has 256 columns, eight threads (one of each warp) to
// every eight columns.  Behind a product of the same call it starts at once and reads dy on the SMs that
// the product's tiles leave idle (dy was complete before the product began); one block then waits for the
// product, so that this kernel ends after it.  As the call's first kernel it waits before it reads.  Bound by the bytes
// of dy and the SMs that are idle: 16384 x 1024 in 23 us alone, under dw's 92.
constexpr int kRun = 512;
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) k_colsum_part(const T* __restrict__ dy, int64_t lddy, int64_t rows, int cols, bool wait_first,
                                                     float* __restrict__ part, void* db, int grad) {
  __shared__ float red[8][256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c0 = blockIdx.x * 256;
  if (wait_first) in_turn();
  for (int64_t run = blockIdx.y; run * kRun < rows; run += gridDim.y) {
    const int64_t end = (run + 1) * kRun < rows ? (run + 1) * kRun : rows;
    float s[8] = {};
    if (VEC) {  // columns c0 + 8 lane ..
      if (c0 + lane * 8 < cols) {
#pragma unroll 8
        for (int64_t r = run * kRun + warp; r < end; r += 8) {
          f2 v[4];
          expand8(load8(dy + r * lddy + c0 + lane * 8), v);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 h = halves(v[i]);
            s[2 * i] += h.x, s[2 * i + 1] += h.y;
          }
        }
      }
    } else {  // columns c0 + lane + 32 i
#pragma unroll 4
      for (int64_t r = run * kRun + warp; r < end; r += 8)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (c0 + lane + 32 * i < cols) s[i] += to_f(dy[r * lddy + c0 + lane + 32 * i]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) red[warp][VEC ? i * 32 + lane : lane + 32 * i] = s[i];
    __syncthreads();
    const int t = threadIdx.x, c = c0 + (VEC ? (t & 31) * 8 + t / 32 : t);
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) v += red[w][t];
    if (c < cols) {
      if (!db) part[run * cols + c] = v;
      else if (grad == ONEBIT_F32) static_cast<float*>(db)[c] = v;
      else if (grad == ONEBIT_F16) static_cast<__half*>(db)[c] = from_f<__half>(v);
      else static_cast<__nv_bfloat16*>(db)[c] = from_f<__nv_bfloat16>(v);
    }
    __syncthreads();
  }
  if (!wait_first && blockIdx.x == 0 && blockIdx.y == 0) in_turn();
}

// Takes the workspace; with `run`, enqueues the work too.
template <typename T>
cudaError_t backward(const onebit_linear_grad_t& a, Space& ws, cudaStream_t s, bool run, bool padded) {
  const int sms = sm_count();
  const ProductShape sx{a.rows, a.in, a.out}, sw{a.out, a.in, a.rows};
  const Kept<T> v{static_cast<const T*>(a.x), a.ldx, a.codes, a.scales, (int)a.in, (int)ceil_div(a.in, kBlock)};
  // act(v) is not in memory yet.  It is rounded to 16 bits for dw's product: the tensor cores take 16-bit operands, and the
  // forward pass rounded the h = act(v) that it multiplied w with the same way, so that this is dw at that h; a second
  // product with what the rounding leaves off would double dw's time for digits that the forward pass did not have.
  const bool computed = a.dw && (a.codes || a.activation != ONEBIT_ACT_NONE);
  const int64_t ldh = pad8(a.in);
  T* h = computed ? ws.take<T>(a.rows * ldh) : nullptr;
  Readable copies;
  Operand dy{a.dy, a.lddy}, w{}, x{h, ldh};
  if (a.dx || a.dw) dy = copies.take(ws, a.dy, a.lddy, a.rows, a.out);
  if (a.dx) w = copies.take(ws, a.w, a.ldw, a.out, a.in);
  if (a.dw && !computed) x = copies.take(ws, a.x, a.ldx, a.rows, a.in);
  cudaError_t err = run ? copies.run(s) : cudaSuccess;
  if (err != cudaSuccess) return err;
  if (a.dx) {
    const ProductPlan plan = plan_product(sx, sms);
    const Partials part = take_partials(ws, plan, a.rows, a.in);
    const T* add = static_cast<const T*>(a.add);
    if (run && plan.splits == 1) {
      const int need = a.codes && (a.activation != ONEBIT_ACT_NONE || h) ? kKeptCodes : a.activation != ONEBIT_ACT_NONE ? kKeptValue : kKeptNone;
      auto go = [&](auto ctas, auto act, auto kept) {
        InputGradEpilogue<T, decltype(act)::value, decltype(kept)::value> e{};
        e.x = make_input<T>(v.x, a.ldx);
        e.codes = a.codes;
        e.scales = a.scales;
        e.blocks = v.blocks;
        e.add = make_input<T>(add, a.ldadd);
        e.act = a.activation;
        e.kept = need;
        e.wide_codes = aligned(a.codes, 32) && a.in % 32 == 0;
        e.vec_codes = aligned(a.codes, 16) && a.in % 16 == 0;
        cudaError_t r = make_output(&e.dx, static_cast<T*>(a.dx), a.rows, a.in, a.lddx);
        if (r == cudaSuccess) r = make_output(&e.h, h, a.rows, a.in, ldh, true);
        return r == cudaSuccess ? run_product_by<decltype(ctas)::value, false, true>(a.dtype, dy, w, sx, plan, e, s) : r;
      };
      using std::integral_constant;
      using Two = integral_constant<int, 2>;
      auto by_act = [&](auto kept) {
        switch (a.activation) {
          case ONEBIT_ACT_RELU: return go(Two{}, integral_constant<int, ONEBIT_ACT_RELU>{}, kept);
          case ONEBIT_ACT_GELU: return go(Two{}, integral_constant<int, ONEBIT_ACT_GELU>{}, kept);
          default: return go(Two{}, integral_constant<int, ONEBIT_ACT_GELU_TANH>{}, kept);
        }
      };
      using None = integral_constant<int, ONEBIT_ACT_NONE>;
      using Codes = integral_constant<int, kKeptCodes>;
      if (plan.ctas == 1) err = go(integral_constant<int, 1>{}, integral_constant<int, kAny>{}, integral_constant<int, kAny>{});
      else if (need == kKeptNone) err = go(Two{}, None{}, integral_constant<int, kKeptNone>{});
      else if (need == kKeptValue) err = by_act(integral_constant<int, kKeptValue>{});
      else if (a.activation == ONEBIT_ACT_NONE) err = go(Two{}, None{}, Codes{});
      else err = by_act(Codes{});
    } else if (run) {
      PlainEpilogue<float> to{};
      err = to_partials(&to, part, a.in);
      if (err == cudaSuccess) err = run_product<false, true>(a.dtype, dy, w, sx, plan, to, s);
      if (err == cudaSuccess)
        err = launch_after(k_finish_dx<T>, flat_grid(a.rows * (part.ld / 4), 256), 256, s, part, a.rows, (int)a.in, v, a.activation, add, a.ldadd,
                           static_cast<T*>(a.dx), a.lddx, h, ldh);
    }
    if (err != cudaSuccess) return err;
  } else if (computed && run) {
    err = launch_after(k_operand<T>, flat_grid(a.rows * a.in, 256), 256, s, v, a.rows, (int)a.in, a.activation, h, ldh);
    if (err != cudaSuccess) return err;
  }
  if (a.dw) {
    const ProductPlan plan = plan_product(sw, sms);
    const Partials part = take_partials(ws, plan, a.out, a.in);
    if (run)
      with_grad(a.grad_dtype, a.dw, [&](auto* g) {
        using G = std::remove_pointer_t<decltype(g)>;
        if (plan.splits == 1) {
          PlainEpilogue<G> e{};
          err = make_output(&e.out, g, a.out, a.in, a.in);
          if (err == cudaSuccess) err = run_product<true, true>(a.dtype, dy, x, sw, plan, e, s);
        } else {
          PlainEpilogue<float> to{};
          err = to_partials(&to, part, a.in);
          if (err == cudaSuccess) err = run_product<true, true>(a.dtype, dy, x, sw, plan, to, s);
          if (err == cudaSuccess) err = launch_after(k_finish_dw<G>, flat_grid(a.out * (part.ld / 4), 256), 256, s, part, a.out, (int)a.in, g);
        }
      });
    if (err != cudaSuccess) return err;
  }
  if (a.db) {
    const int64_t chunks = ceil_div(a.rows, kRun);
    float* part = chunks > 1 ? ws.take<float>(chunks * a.out) : nullptr;
    void* whole = chunks > 1 ? nullptr : a.db;
    if (run) {
      const T* p = static_cast<const T*>(dy.p);
      const dim3 grid((unsigned)ceil_div(a.out, 256), (unsigned)(chunks < 65535 ? chunks : 65535));
      const bool first = !a.dx && !a.dw;
      // eight columns at a time where the last eight lie inside the row (a realigned copy is padded to them)
      err = vec16(p, dy.ld) && (a.out % 8 == 0 || padded || p != a.dy)
                ? launch_after(k_colsum_part<T, true>, grid, 256, s, p, dy.ld, a.rows, (int)a.out, first, part, whole, a.grad_dtype)
                : launch_after(k_colsum_part<T, false>, grid, 256, s, p, dy.ld, a.rows, (int)a.out, first, part, whole, a.grad_dtype);
      if (err == cudaSuccess && chunks > 1) err = sum_parts(a.grad_dtype, part, chunks, a.out, a.out, a.db, nullptr, s);
      if (err != cudaSuccess) return err;
    }
  }
  return err;
}
onebit_status_t backward_ok(const onebit_linear_grad_t* a) {
  if (!a) return fail(ONEBIT_ERR_INVALID_ARG, "the arguments are NULL");
  onebit_status_t st = linear_shape_ok(a->rows, a->in, a->out, a->dtype, a->activation);
  if (st != ONEBIT_OK) return st;
  if (!dtype_ok(a->grad_dtype)) return fail(ONEBIT_ERR_INVALID_ARG, "grad_dtype is not one of f32, f16, bf16");
  if (!a->codes != !a->scales) return fail(ONEBIT_ERR_INVALID_ARG, "a checkpoint needs codes and scales");
  if (a->x && a->codes) return fail(ONEBIT_ERR_INVALID_ARG, "the input is x or its checkpoint, not both");
  if (a->lddy < a->out || (a->x && a->ldx < a->in) || (a->dx && (a->ldw < a->in || a->lddx < a->in || (a->add && a->ldadd < a->in))))
    return fail(ONEBIT_ERR_INVALID_ARG, "a row stride below the columns");
  if (a->rows > 0) {
    if ((a->dx || a->dw || a->db) && !a->dy) return fail(ONEBIT_ERR_INVALID_ARG, "a NULL buffer");
    if (a->dx && !a->w) return fail(ONEBIT_ERR_INVALID_ARG, "dx needs the weight");
    if ((a->dw || (a->dx && a->activation != ONEBIT_ACT_NONE)) && !a->x && !a->codes)
      return fail(ONEBIT_ERR_INVALID_ARG, "dw and the activation's derivative need x or its checkpoint");
  }
  const uintptr_t g = (uintptr_t)dtype_size(a->grad_dtype);
  if (!aligned(a->dy, 2) || !aligned(a->x, 2) || !aligned(a->w, 2) || !aligned(a->add, 2) || !aligned(a->dx, 2) ||
      !aligned(a->scales, 4) || !aligned(a->dw, g) || !aligned(a->db, g))
    return fail(ONEBIT_ERR_INVALID_ARG, "a buffer is not aligned to its type");
  return ONEBIT_OK;
}

}  // namespace

cudaError_t linear_backward(const onebit_linear_grad_t& a, Space& ws, cudaStream_t s, bool run, bool padded) {
  return a.dtype == ONEBIT_F16 ? backward<__half>(a, ws, s, run, padded) : backward<__nv_bfloat16>(a, ws, s, run, padded);
}

}  // namespace layers
}  // namespace onebit

using namespace onebit::layers;

extern "C" onebit_status_t onebit_linear_backward_workspace(const onebit_linear_grad_t* a, size_t* bytes) {
  onebit_status_t st = backward_ok(a);
  if (st != ONEBIT_OK) return st;
  if (!bytes) return fail(ONEBIT_ERR_INVALID_ARG, "bytes is NULL");
  Space ws{nullptr};
  if (a->rows > 0) linear_backward(*a, ws, nullptr, false);
  *bytes = (size_t)ws.used;
  return ONEBIT_OK;
}

extern "C" onebit_status_t onebit_linear_backward(const onebit_linear_grad_t* a, void* workspace,
                                                  size_t workspace_bytes, onebit_stream_t stream) {
  size_t need = 0;
  onebit_status_t st = onebit_linear_backward_workspace(a, &need);
  if (st != ONEBIT_OK) return st;
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256)))
    return fail(ONEBIT_ERR_WORKSPACE, "the workspace is too small or not 256-byte aligned");
  const int64_t blocks = ceil_div(a->in, kBlock), g = dtype_size(a->grad_dtype);
  if (!disjoint({matrix(a->dy, a->rows, a->lddy, a->out, 2), matrix(a->x, a->rows, a->ldx, a->in, 2),
                 span_of(a->codes, a->rows * a->in), span_of(a->scales, a->rows * blocks * 4),
                 matrix(a->w, a->out, a->ldw, a->in, 2), matrix(a->add, a->rows, a->ldadd, a->in, 2)},
                {matrix(a->dx, a->rows, a->lddx, a->in, 2), span_of(a->dw, a->out * a->in * g),
                 span_of(a->db, a->out * g), span_of(workspace, (int64_t)need)}))
    return fail(ONEBIT_ERR_INVALID_ARG, "an output overlaps another buffer");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (a->rows > 0) {
    Space ws{static_cast<char*>(workspace)};
    e = linear_backward(*a, ws, s, true);
  } else {  // no tokens: the parameters' gradients are 0
    if (a->dw) e = cudaMemsetAsync(a->dw, 0, (size_t)(a->out * a->in * g), s);
    if (a->db && e == cudaSuccess) e = cudaMemsetAsync(a->db, 0, (size_t)(a->out * g), s);
  }
  return e == cudaSuccess ? ONEBIT_OK : cuda_fail(e, "onebit_linear_backward");
}
