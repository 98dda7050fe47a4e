// Backward under score rules, instances for head size 128 (bf16 / fp32 gradients).
#include "fa_rules_bwd_kernel.cuh"

namespace fa {
cudaError_t launch_bwd_rules_128(const BwdRulesParams& p, fa_dtype grad_dtype, cudaStream_t st)
{
    return launch_bwd_rules_d<128>(p, grad_dtype, st);
}
}  // namespace fa
