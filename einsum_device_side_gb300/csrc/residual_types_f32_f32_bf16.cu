// residual_types_f32_f32_bf16.cu -- the kernels of residual_norm.cuh for one set of types.
#define TROP_TU 12  // the id of residual_norm.cuh in a bounds-violation record
#include "residual_norm.cuh"

namespace trop {
template int residual_forward<float, float, bf16>(ResJob, int, cudaStream_t);
template int residual_backward<float, float, bf16, false>(ResJob, JoinJob, int, cudaStream_t);
template int residual_backward<float, float, bf16, true>(ResJob, JoinJob, int, cudaStream_t);
}  // namespace trop
