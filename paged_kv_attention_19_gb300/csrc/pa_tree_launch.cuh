// pa_tree_launch.cuh -- launches of the tree attention's kernels, instantiated once per cache format by
// pa_tree_{bf16,fp8,nvfp4}.cu (one translation unit each, built in parallel).
#pragma once

#include "pa_tree.cuh"

namespace pa {

struct TreeLaunch {
  const CUtensorMap &tm_k, &tm_v, &tm_q;
  const TreeArgs &a;
  uint32_t *status;  // the workspace's status word
  int D, QT;
};

cudaError_t launch_tree_bf16(const TreeLaunch &l, cudaStream_t stream);
cudaError_t launch_tree_fp8(const TreeLaunch &l, cudaStream_t stream);
cudaError_t launch_tree_nvfp4(const TreeLaunch &l, cudaStream_t stream);

template <typename K, typename... A>
cudaError_t launch_pdl(K kernel, dim3 grid, int threads, int smem, cudaStream_t stream, A &&...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int D, int FMT, int QT>
cudaError_t launch_tree(const TreeLaunch &l, cudaStream_t stream) {
  using C = TreeCfg<D, FMT, QT>;
  const TreeArgs &a = l.a;
  // (made at every call: the attribute is the device's, and costs less than to remember where it is set)
  cudaError_t e = cudaFuncSetAttribute(tree_split_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, TreeSmem<C>::BYTES);
  if (e != cudaSuccess) return e;
  e = launch_pdl(tree_split_kernel<C>, dim3((unsigned)a.nparts), C::THREADS, TreeSmem<C>::BYTES, stream,
                 l.tm_k, l.tm_v, l.tm_q, a);
  if (e != cudaSuccess) return e;
  const int groups = (tree_max_rows(a, QT) + combine_rows(D) - 1) / combine_rows(D);
  const dim3 grid((unsigned)a.nparts, (unsigned)(groups < kCombineBlocks ? groups : kCombineBlocks));
  return launch_pdl(tree_combine_kernel<D, QT>, grid, kCombineThreads, 0, stream, a, l.status);
}

template <int FMT>
cudaError_t launch_tree_any(const TreeLaunch &l, cudaStream_t stream) {
  switch (l.D) {
    case 64: return l.QT == 2 ? launch_tree<64, FMT, 2>(l, stream) : launch_tree<64, FMT, 1>(l, stream);
    case 128: return l.QT == 2 ? launch_tree<128, FMT, 2>(l, stream) : launch_tree<128, FMT, 1>(l, stream);
    default: return launch_tree<256, FMT, 1>(l, stream);
  }
}

}  // namespace pa
