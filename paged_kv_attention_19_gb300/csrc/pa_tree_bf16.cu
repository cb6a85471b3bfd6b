// pa_tree_bf16.cu -- the tree attention over bf16 pools.
#include "pa_tree_launch.cuh"

namespace pa {

cudaError_t launch_tree_bf16(const TreeLaunch &l, cudaStream_t stream) {
  return launch_tree_any<TREE_BF16>(l, stream);
}

}  // namespace pa
