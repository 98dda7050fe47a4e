// Decode behind a shared prefix (fa_tree_kernel, SHARED), head size 32.
#include "fa_tree_kernel.cuh"

namespace fa {
cudaError_t launch_prefix_32(const PrefixParams& p, cudaStream_t st) { return launch_prefix_d<32>(p, st); }
}  // namespace fa
