// pa_host.h -- what the host sides of the attention calls share: alignment, powers of two, overlaps, launches, tensor
// maps, the device's size.
#pragma once

#include <cstddef>
#include <cstdint>
#include <mutex>

#include <cuda_runtime.h>
#include <cudaTypedefs.h>

namespace pa {

inline bool aligned_to(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }
inline bool is_pow2(int x) { return x > 0 && (x & (x - 1)) == 0; }
inline int ilog2(int x) {
  int l = 0;
  while ((1 << l) < x) ++l;
  return l;
}
inline size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Do [p, p + np) and [q, q + nq) share a byte?
inline bool overlap(const void *p, size_t np, const void *q, size_t nq) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return a < b + nq && b < a + np;
}

// A launch that may begin while the stream's previous kernel ends; cluster > 0: in clusters of so many CTAs.
template <typename Args>
cudaError_t launch(void (*kernel)(Args), dim3 grid, int threads, size_t smem, int cluster, const Args &a,
                   cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 0 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// A map of RANK dimensions (the first one contiguous, the others dense or so many bytes apart): bf16 values with the 128-byte
// swizzle, or bytes.
template <int RANK>
bool encode_map(CUtensorMap *m, const void *base, const cuuint64_t (&dims)[RANK], const cuuint32_t (&box)[RANK], bool bytes,
                const cuuint64_t *apart = nullptr) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t strides[RANK - 1], s = bytes ? 1 : 2;
  cuuint32_t ones[RANK];
  for (int i = 0; i < RANK; ++i) {
    ones[i] = 1u;
    if (i < RANK - 1) strides[i] = s = apart ? apart[i] : s * dims[i];
  }
  return fn(m, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, RANK, const_cast<void *>(base),
            dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
            bytes ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// SMs of the current device; -1: the runtime has no answer.
inline int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return -1;
  return n;
}

}  // namespace pa
