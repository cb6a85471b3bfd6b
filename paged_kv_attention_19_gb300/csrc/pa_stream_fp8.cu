// pa_stream_fp8.cu -- the streams' attention over FP8 pools.
#include "pa_stream_launch.cuh"

namespace pa {

cudaError_t launch_stream_fp8(const StreamLaunch &l, cudaStream_t stream) {
  return launch_stream_any<TREE_FP8>(l, stream);
}

}  // namespace pa
