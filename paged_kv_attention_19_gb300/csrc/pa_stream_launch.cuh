// pa_stream_launch.cuh -- launches of the streams' attention kernels, instantiated once per cache format by
// pa_stream_{bf16,fp8,nvfp4}.cu (one translation unit each, built in parallel).
#pragma once

#include "pa_stream.cuh"
#include "pa_tree_launch.cuh"

namespace pa {

struct StreamLaunch {
  const CUtensorMap &tm_k, &tm_v, &tm_q;
  const StreamArgs &a;
  uint32_t *status;  // the workspace's status word
  int D, QT;
};

cudaError_t launch_stream_bf16(const StreamLaunch &l, cudaStream_t stream);
cudaError_t launch_stream_fp8(const StreamLaunch &l, cudaStream_t stream);
cudaError_t launch_stream_nvfp4(const StreamLaunch &l, cudaStream_t stream);

template <int D, int FMT, int QT>
cudaError_t launch_stream(const StreamLaunch &l, cudaStream_t stream) {
  using C = StreamCfg<D, FMT, QT>;
  const StreamArgs &a = l.a;
  // (made at every call: the attribute is the device's, and costs less than to remember where it is set)
  cudaError_t e = cudaFuncSetAttribute(stream_split_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, StreamSmem<C>::BYTES);
  if (e != cudaSuccess) return e;
  e = launch_pdl(stream_split_kernel<C>, dim3((unsigned)a.nparts), C::THREADS, StreamSmem<C>::BYTES, stream, l.tm_k, l.tm_v,
                 l.tm_q, a);
  if (e != cudaSuccess) return e;
  // the rows that an item can have: of a single tile those that it holds
  const int rows = QT == 2 ? 2 * kTreeRows : a.G * (a.qt < a.max_query ? a.qt : a.max_query);
  const int blocks = (rows + combine_rows(D) - 1) / combine_rows(D);
  const dim3 grid((unsigned)a.nparts, (unsigned)(blocks < kCombineBlocks ? blocks : kCombineBlocks));
  return launch_pdl(stream_combine_kernel<D, QT>, grid, kCombineThreads, 0, stream, a, l.status);
}

template <int FMT>
cudaError_t launch_stream_any(const StreamLaunch &l, cudaStream_t stream) {
  switch (l.D) {
    case 64: return l.QT == 2 ? launch_stream<64, FMT, 2>(l, stream) : launch_stream<64, FMT, 1>(l, stream);
    case 128: return l.QT == 2 ? launch_stream<128, FMT, 2>(l, stream) : launch_stream<128, FMT, 1>(l, stream);
    default: return launch_stream<256, FMT, 1>(l, stream);
  }
}

}  // namespace pa
