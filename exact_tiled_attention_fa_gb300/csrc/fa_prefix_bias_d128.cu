// Decode behind a shared prefix (fa_tree_kernel, SHARED), head size 128, scores with a bias.
#include "fa_tree_kernel.cuh"

namespace fa {
template <>
cudaError_t launch_prefix<128, 2>(const PrefixParams& p, cudaStream_t st) { return launch_prefix_d<128, 2>(p, st); }
}  // namespace fa
