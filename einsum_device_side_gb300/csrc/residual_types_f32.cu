// residual_types_f32.cu -- the kernels of residual_norm.cuh for one set of types.
#define TROP_TU 12  // the id of residual_norm.cuh in a bounds-violation record
#include "residual_norm.cuh"

namespace trop {
template int residual_forward<float, float, float>(ResJob, int, cudaStream_t);
template int residual_backward<float, float, float, false>(ResJob, JoinJob, int, cudaStream_t);
template int residual_backward<float, float, float, true>(ResJob, JoinJob, int, cudaStream_t);
}  // namespace trop
