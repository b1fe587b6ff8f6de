// residual_norm_f16.cu -- the residual norm's kernels for one type (a file each: they compile side by side).
#include "residual_norm.cuh"

namespace onebit {
namespace layers {

template cudaError_t rn_forward<__half>(ResidualForward, cudaStream_t);
template cudaError_t rn_backward<__half>(ResidualBackward, const ParamGrads&, int32_t, char*, int64_t*, cudaStream_t, bool);

}  // namespace layers
}  // namespace onebit
