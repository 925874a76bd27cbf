// Norm over groups: the calls, and the kernels for float32.
#include "group_norm.cuh"

namespace mixer {

cudaError_t run_group_norm_f32(const GroupNormParams &p, bool bwd, cudaStream_t s) { return run_t<float>(p, plan_of(p, false, bwd), bwd, s); }

size_t group_norm_part_floats(const GroupNormParams &p, bool bf16_) {
    return (size_t)plan_of(p, bf16_, true).parts * 2 * (p.shared ? p.C : (size_t)p.G * p.C);
}

cudaError_t launch_group_norm_fwd(const GroupNormParams &p, bool bf16_, cudaStream_t s) {
    return bf16_ ? run_group_norm_bf16(p, false, s) : run_group_norm_f32(p, false, s);
}

cudaError_t launch_group_norm_bwd(const GroupNormParams &p, bool bf16_, cudaStream_t s) {
    const cudaError_t e = bf16_ ? run_group_norm_bf16(p, true, s) : run_group_norm_f32(p, true, s);
    if (e != cudaSuccess || !p.part) return e;
    const long long cols = p.shared ? p.C : (long long)p.G * p.C;
    return launch_sum_rows(p.part, plan_of(p, bf16_, true).parts, SumOut{p.dweight, cols, p.w_bf16}, SumOut{p.dbias, cols, p.w_bf16}, s);
}

}  // namespace mixer
