// pa_stream_nvfp4.cu -- the streams' attention over NVFP4 pools.
#include "pa_stream_launch.cuh"

namespace pa {

cudaError_t launch_stream_nvfp4(const StreamLaunch &l, cudaStream_t stream) {
  return launch_stream_any<TREE_NVFP4>(l, stream);
}

}  // namespace pa
