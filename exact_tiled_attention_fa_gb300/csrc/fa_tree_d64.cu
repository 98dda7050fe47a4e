// Tree decode, head size 64.
#include "fa_tree_kernel.cuh"

namespace fa {
cudaError_t launch_tree_64(const TreeParams& p, cudaStream_t st) { return launch_tree_d<64>(p, st); }
}  // namespace fa
