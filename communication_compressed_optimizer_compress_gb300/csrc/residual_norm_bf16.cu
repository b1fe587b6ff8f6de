// residual_norm_bf16.cu -- the residual norm's kernels for one type (a file each: they compile side by side).
#include "residual_norm.cuh"

namespace onebit {
namespace layers {

template cudaError_t rn_forward<__nv_bfloat16>(ResidualForward, cudaStream_t);
template cudaError_t rn_backward<__nv_bfloat16>(ResidualBackward, const ParamGrads&, int32_t, char*, int64_t*, cudaStream_t, bool);

}  // namespace layers
}  // namespace onebit
