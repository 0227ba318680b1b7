// residual_types_bf16.cu -- the kernels of residual_norm.cuh for one set of types.
#define TROP_TU 12  // the id of residual_norm.cuh in a bounds-violation record
#include "residual_norm.cuh"

namespace trop {
template int residual_forward<bf16, bf16, bf16>(ResJob, int, cudaStream_t);
template int residual_backward<bf16, bf16, bf16, false>(ResJob, JoinJob, int, cudaStream_t);
template int residual_backward<bf16, bf16, bf16, true>(ResJob, JoinJob, int, cudaStream_t);
}  // namespace trop
