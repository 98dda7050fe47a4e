// Tree decode, head size 128.
#include "fa_tree_kernel.cuh"

namespace fa {
cudaError_t launch_tree_128(const TreeParams& p, cudaStream_t st) { return launch_tree_d<128>(p, st); }
}  // namespace fa
