// Forward under score rules, instances for head size 64 (bf16 / fp32 output).
#include "fa_rules_fwd_kernel.cuh"

namespace fa {
cudaError_t launch_fwd_rules_64(const FwdRulesParams& p, fa_dtype o_dtype, cudaStream_t st)
{
    return launch_fwd_rules_d<64>(p, o_dtype, st);
}
}  // namespace fa
