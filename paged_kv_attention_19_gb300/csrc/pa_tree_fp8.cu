// pa_tree_fp8.cu -- the tree attention over FP8 E4M3 pools.
#include "pa_tree_launch.cuh"

namespace pa {

cudaError_t launch_tree_fp8(const TreeLaunch &l, cudaStream_t stream) {
  return launch_tree_any<TREE_FP8>(l, stream);
}

}  // namespace pa
