// gated_common.cuh -- what the gated linear layer's forward and backward pass share: how g and u are kept, and their
// activation outside the products' epilogues.
#pragma once

#include "linear_common.cuh"

namespace onebit {
namespace layers {

// (activation, derivative), with silu beside those of the linear layer
__device__ __forceinline__ float2 gate_both(int act, float g) { return act == ONEBIT_ACT_SILU ? act_one<ONEBIT_ACT_SILU>(g) : act_both(act, g); }

inline onebit_status_t gated_shape_ok(int64_t rows, int64_t a, int64_t inner, int32_t dtype, int32_t act) {
  if (inner > kMaxCols / 2) return fail(ONEBIT_ERR_UNSUPPORTED, "an inner width above 2^23");
  return linear_shape_ok(rows, a, inner, dtype, act == ONEBIT_ACT_SILU ? ONEBIT_ACT_NONE : act);
}
// all four of the checkpoints or none
inline bool checkpoints_whole(const void* gc, const void* gs, const void* uc, const void* us) { return !gc == !gs && !gc == !uc && !gc == !us; }

}  // namespace layers
}  // namespace onebit
