// gated_forward.cu -- the gated linear layer's forward pass: both projections in one matrix product, activation,
// gating and what is kept.  See include/onebit_layers.h for the formulas.
#include "few_rows.cuh"
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

// The epilogue over the sums z of a cut contraction, one warp per 64 columns of a row of h (a checkpoint's block), elements side by side.
// Bound by the sums' bytes, out of the L2: 512 x 4096 x 256 in four parts.
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

// Up to 32 rows, as generation meets them: the few-rows product (few_rows.cuh) with two weights to a column, the gate's and
// the up projection's, whose sums meet in shared memory.  Bound by the weights' bytes and a launch's latency: a warp asks for kAhead
// steps of both weights, and of x where it is up to eight rows, before it multiplies any; 128 registers a thread hold them.  One row of
// 4096 -> 12288 34 us, where the weights alone are 30 (with 64 registers, which spill, a sixth longer); of 1024 -> 4096, weights in HBM, 4.4 us a
// call, 5.2 without sending for them before the turn.  Nine rows and more are bound by x, all of which every block of eight columns reads: 32 rows
// of 4096 -> 12288 take 50 us, 403 MB out of the L2 beside the weights' 201, with L1's data pipe at 64% (one row 32%); sixteen 39.
struct FewGatedArgs {
  const void* x;
  int64_t ldx;
  const void* w;
  int64_t ldw;
  const float* bias;
  void* h;
  int64_t ldh;
  int rows, in, inner, act;
};
// HALVES of eight rows: 1, 2 or 4
template <typename T, int HALVES>
__global__ void __launch_bounds__(kFewThreads, 2) k_few_rows_gated(const FewGatedArgs A) {
  constexpr int kSplits = 8, kAhead = 4, M = HALVES == 4 ? 2 : 1;
  __shared__ float part[kSplits][2][HALVES * 8][9];
  const int lane = threadIdx.x & 31, split = threadIdx.x >> 5;
  const int n = lane >> 2, q = lane & 3;
  const int col = blockIdx.x * 8 + n;
  const int steps = (A.in + 31) / 32, per = (steps + kSplits - 1) / kSplits;
  const int s1 = split * per + per < steps ? split * per + per : steps;
  const T* w = static_cast<const T*>(A.w) + (int64_t)(col < A.inner ? col : 0) * A.ldw + q * 8;
  const T* x = static_cast<const T*>(A.x) + (int64_t)n * A.ldx + q * 8;
  const int64_t up = (int64_t)A.inner * A.ldw;
  float d[2][M][4] = {};
  const uint4 zero = make_uint4(0, 0, 0, 0);
  // the first steps' weights (two lines of a row) on their way to the L2 beside the kernel before, whatever it writes
  const int k0 = split * per * 32 + (q & 1) * 64;
  if (col < A.inner && k0 < A.in) asm volatile("prefetch.global.L2 [%0];" ::"l"(w - q * 8 + (q & 2 ? up : 0) + k0));
  in_turn();
  for (int s = split * per; s < s1; s += kAhead) {
    uint4 b[kAhead][2], a[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int k = (s + i) * 32;
      const bool in = s + i < s1 && k + q * 8 < A.in;
      b[i][0] = in && col < A.inner ? __ldg(reinterpret_cast<const uint4*>(w + k)) : zero;
      b[i][1] = in && col < A.inner ? __ldg(reinterpret_cast<const uint4*>(w + up + k)) : zero;
      if (HALVES == 1) a[i] = in && n < A.rows ? __ldg(reinterpret_cast<const uint4*>(x + k)) : zero;
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int k = (s + i) * 32;
      const bool in = s + i < s1 && k + q * 8 < A.in;
#pragma unroll
      for (int m = 0; m < M; ++m) {
        auto row = [&](int r) { return in && r + n < A.rows ? __ldg(reinterpret_cast<const uint4*>(x + r * A.ldx + k)) : zero; };
        const uint4 lo = HALVES == 1 ? a[i] : row(16 * m), hi = HALVES == 1 ? zero : row(16 * m + 8);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          mma_16x8x16<T>(d[p][m], lo.x, hi.x, lo.y, hi.y, b[i][p].x, b[i][p].y);
          mma_16x8x16<T>(d[p][m], lo.z, hi.z, lo.w, hi.w, b[i][p].z, b[i][p].w);
        }
      }
    }
  }
#pragma unroll
  for (int p = 0; p < 2; ++p)
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int i = 0; i < (HALVES == 1 ? 2 : 4); ++i) part[split][p][m * 16 + n + 8 * (i / 2)][2 * q + (i & 1)] = d[p][m][i];
  __syncthreads();
  const int r = threadIdx.x / 8, j = threadIdx.x % 8, c = blockIdx.x * 8 + j;
  if (r >= A.rows || c >= A.inner) return;  // (at most 32 rows: a thread has one value)
  float g = part[0][0][r][j], u = part[0][1][r][j];
#pragma unroll
  for (int s = 1; s < kSplits; ++s) g += part[s][0][r][j], u += part[s][1][r][j];
  if (A.bias) g += __ldg(A.bias + c), u += __ldg(A.bias + A.inner + c);
  static_cast<T*>(A.h)[r * A.ldh + c] = from_f<T>(gate_both(A.act, g).x * u);
}
// Few rows, on 16 bytes, and nothing kept.
inline bool few_rows(const onebit_gated_linear_t& a) {
  return a.rows <= kFewRows && !a.z && !a.gate_codes && a.in % 8 == 0 && vec16(a.x, a.ldx) && vec16(a.w, a.ldw);
}
template <typename T>
cudaError_t run_few_rows(const onebit_gated_linear_t& a, cudaStream_t s) {
  const FewGatedArgs f{a.x, a.ldx, a.w, a.ldw, a.bias, a.h, a.ldh, (int)a.rows, (int)a.in, (int)a.inner, a.activation};
  const unsigned grid = (unsigned)ceil_div(a.inner, 8);
  if (a.rows <= 8) return launch_after(k_few_rows_gated<T, 1>, grid, kFewThreads, s, f);
  return a.rows <= 16 ? launch_after(k_few_rows_gated<T, 2>, grid, kFewThreads, s, f) : launch_after(k_few_rows_gated<T, 4>, grid, kFewThreads, s, f);
}

// Takes the workspace; with `run`, enqueues the work too.
template <typename T>
cudaError_t forward(const onebit_gated_linear_t& a, Space& ws, cudaStream_t s, bool run) {
  if (few_rows(a)) return run ? run_few_rows<T>(a, s) : cudaSuccess;
  const ProductShape shape{a.rows, 2 * a.inner, a.in};
  const ProductPlan plan = plan_product(shape, sm_count());
  Readable copies;
  const Operand x = copies.take(ws, a.x, a.ldx, a.rows, a.in), w = copies.take(ws, a.w, a.ldw, 2 * a.inner, a.in);
  // the bias's halves as rows of 16-bit words: they start on 16 bytes, or their realigned copies do
  const bool in_epilogue = plan.splits == 1 && a.bias;
  const Operand bias = in_epilogue ? copies.take(ws, a.bias, 2 * a.inner, 2, 2 * a.inner) : Operand{};
  const Partials part = take_partials(ws, plan, a.rows, 2 * a.inner);
  if (!run) return cudaSuccess;
  cudaError_t err = copies.run(s);
  if (err != cudaSuccess) return err;
  const int64_t blocks = ceil_div(a.inner, kBlock);
  if (plan.splits == 1) {
    auto go = [&](auto ctas, auto act, auto keep) {
      GatedEpilogue<T, decltype(act)::value, decltype(keep)::value> e{};
      T* z = static_cast<T*>(a.z);
      if (in_epilogue) e.gate_bias = static_cast<const float*>(bias.p), e.up_bias = e.gate_bias + bias.ld / 2;
      e.gate_scales = a.gate_scales, e.up_scales = a.up_scales;
      e.blocks = (int)blocks, e.act = a.activation, e.keep = a.z ? kKeptValue : a.gate_codes ? kKeptCodes : kKeptNone;
      cudaError_t r = make_output(&e.h, static_cast<T*>(a.h), a.rows, a.inner, a.ldh);
      if (r == cudaSuccess) r = make_output(&e.gate, z, a.rows, a.inner, a.ldz);
      if (r == cudaSuccess) r = make_output(&e.up, z ? z + a.inner : nullptr, a.rows, a.inner, a.ldz);
      if (r == cudaSuccess) r = make_output(&e.gate_codes, a.gate_codes, a.rows, a.inner, a.inner);
      if (r == cudaSuccess) r = make_output(&e.up_codes, a.up_codes, a.rows, a.inner, a.inner);
      return r == cudaSuccess ? run_product_by<decltype(ctas)::value, false, false>(a.dtype, x, w, shape, plan, e, s) : r;
    };
    using std::integral_constant;
    using Any = integral_constant<int, kAny>;
    if (plan.ctas == 1) return go(integral_constant<int, 1>{}, Any{}, Any{});
    auto by_act = [&](auto keep) {
      integral_constant<int, 2> two;
      switch (a.activation) {
        case ONEBIT_ACT_GELU: return go(two, integral_constant<int, ONEBIT_ACT_GELU>{}, keep);
        case ONEBIT_ACT_GELU_TANH: return go(two, integral_constant<int, ONEBIT_ACT_GELU_TANH>{}, keep);
        case ONEBIT_ACT_SILU: return go(two, integral_constant<int, ONEBIT_ACT_SILU>{}, keep);
        default: return go(two, Any{}, keep);
      }
    };
    return a.z ? by_act(integral_constant<int, kKeptValue>{})
           : a.gate_codes ? by_act(integral_constant<int, kKeptCodes>{}) : by_act(integral_constant<int, kKeptNone>{});
  }
  PlainEpilogue<float> to{};
  err = to_partials(&to, part, 2 * a.inner);
  if (err == cudaSuccess) err = run_product<false, false>(a.dtype, x, w, shape, plan, to, s);
  if (err != cudaSuccess) return err;
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
