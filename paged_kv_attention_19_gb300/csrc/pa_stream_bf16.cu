// pa_stream_bf16.cu -- the streams' attention over bf16 pools.
#include "pa_stream_launch.cuh"

namespace pa {

cudaError_t launch_stream_bf16(const StreamLaunch &l, cudaStream_t stream) {
  return launch_stream_any<TREE_BF16>(l, stream);
}

}  // namespace pa
