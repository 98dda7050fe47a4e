// fa_rules_ranges.cu -- the queries' intervals of keys (fa_rules_ranges.cuh), before a forward pass over documents.  (The
// keys' intervals of queries are made by the backward's preparation, fa_bwd.cu.)
#include "fa_rules_ranges.cuh"

namespace fa {

__global__ void __launch_bounds__(kRangeThreads) fa_rules_ranges_kernel(const RangesParams p)
{
    grid_dependency_wait();
    grid_launch_dependents();
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.counter = 0;
    rules_ranges<false>(p, static_cast<int>(blockIdx.x));
}

cudaError_t launch_rules_ranges(const RangesParams& p, cudaStream_t st)
{
    const long long ctas = static_cast<long long>(p.B) * p.tiles;
    if (ctas <= 0 || ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
    return launch_pdl(fa_rules_ranges_kernel, static_cast<unsigned>(ctas), kRangeThreads, 0, st, p);
}

}  // namespace fa
