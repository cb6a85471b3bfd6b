// pa_tree_nvfp4.cu -- the tree attention over NVFP4 pools.
#include "pa_tree_launch.cuh"

namespace pa {

cudaError_t launch_tree_nvfp4(const TreeLaunch &l, cudaStream_t stream) {
  return launch_tree_any<TREE_NVFP4>(l, stream);
}

}  // namespace pa
