// The EXT forms of the draft-tree kernel for heads of 64 channels: a translation unit of its own.
#include "sa_tree_kernel.cuh"

namespace sa {

cudaError_t launch_tree_ext64(TreeArgs& a, bool kv_bf16, int rows, cudaStream_t s) { return launch_tree_ext_d<64>(a, kv_bf16, rows, s); }

}  // namespace sa
