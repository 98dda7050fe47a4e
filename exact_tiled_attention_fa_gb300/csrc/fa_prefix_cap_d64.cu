// Decode behind a shared prefix (fa_tree_kernel, SHARED), head size 64, scores with a cap.
#include "fa_tree_kernel.cuh"

namespace fa {
template <>
cudaError_t launch_prefix<64, 1>(const PrefixParams& p, cudaStream_t st) { return launch_prefix_d<64, 1>(p, st); }
}  // namespace fa
