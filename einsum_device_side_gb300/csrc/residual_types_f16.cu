// residual_types_f16.cu -- the kernels of residual_norm.cuh for one set of types.
#define TROP_TU 12  // the id of residual_norm.cuh in a bounds-violation record
#include "residual_norm.cuh"

namespace trop {
template int residual_forward<__half, __half, __half>(ResJob, int, cudaStream_t);
template int residual_backward<__half, __half, __half, false>(ResJob, JoinJob, int, cudaStream_t);
template int residual_backward<__half, __half, __half, true>(ResJob, JoinJob, int, cudaStream_t);
}  // namespace trop
