// Backward under score rules, instances for head size 64 (bf16 / fp32 gradients).
#include "fa_rules_bwd_kernel.cuh"

namespace fa {
cudaError_t launch_bwd_rules_64(const BwdRulesParams& p, fa_dtype grad_dtype, cudaStream_t st)
{
    return launch_bwd_rules_d<64>(p, grad_dtype, st);
}
}  // namespace fa
