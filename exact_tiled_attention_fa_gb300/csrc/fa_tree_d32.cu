// Tree decode, head size 32.
#include "fa_tree_kernel.cuh"

namespace fa {
cudaError_t launch_tree_32(const TreeParams& p, cudaStream_t st) { return launch_tree_d<32>(p, st); }
}  // namespace fa
