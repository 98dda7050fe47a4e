// Forward and backward under score rules, head size 64, scores with no rules (bf16 / fp32 output).
#include "fa_rules_bwd_kernel.cuh"
#include "fa_rules_fwd_kernel.cuh"

namespace fa {
template <>
cudaError_t launch_fwd_rules<64, 0>(const FwdRulesParams& p, fa_dtype o_dtype, cudaStream_t st)
{
    return launch_fwd_rules_d<64, 0>(p, o_dtype, st);
}
template <>
cudaError_t launch_bwd_rules<64, 0>(const BwdRulesParams& p, fa_dtype grad_dtype, cudaStream_t st)
{
    return launch_bwd_rules_d<64, 0>(p, grad_dtype, st);
}
}  // namespace fa
