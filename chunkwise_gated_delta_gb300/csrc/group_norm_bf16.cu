// Norm over groups: the kernels for bfloat16.
#include "group_norm.cuh"

namespace mixer {

cudaError_t run_group_norm_bf16(const GroupNormParams &p, bool bwd, cudaStream_t s) { return run_t<bf16>(p, plan_of(p, true, bwd), bwd, s); }

}  // namespace mixer
