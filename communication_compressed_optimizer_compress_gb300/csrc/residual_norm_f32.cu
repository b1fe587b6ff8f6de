// residual_norm_f32.cu -- the residual norm's kernels for one type (a file each: they compile side by side).
#include "residual_norm.cuh"

namespace onebit {
namespace layers {

template cudaError_t rn_forward<float>(ResidualForward, cudaStream_t);
template cudaError_t rn_backward<float>(ResidualBackward, const ParamGrads&, int32_t, char*, int64_t*, cudaStream_t, bool);

}  // namespace layers
}  // namespace onebit
