// Host-side pieces shared by the expert-layer calls (route.cu, combine.cu,
// w4_matvec.cu).  Host code only.
#pragma once

#include "host.cuh"

namespace arn {

inline bool aligned_to(const void *p, uintptr_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

inline int type_size(int type) {
  return type == AR_TYPE_F32 ? 4 : type == AR_TYPE_BF16 || type == AR_TYPE_F16 ? 2 : 0;
}

// A launch with programmatic stream serialization (every kernel of the
// library waits for the previous grid itself) and, for `cluster` > 1, as
// thread-block clusters.
template <typename Args>
inline cudaError_t launch_pdl(void (*kernel)(Args), const Args &args, int64_t grid, int threads,
                              size_t smem, int cluster, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  int na = 0;
  if (cluster > 1) {
    attr[na].id = cudaLaunchAttributeClusterDimension;
    attr[na].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[na].val.clusterDim.y = 1;
    attr[na].val.clusterDim.z = 1;
    ++na;
  }
  attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[na].val.programmaticStreamSerializationAllowed = 1;
  ++na;
  cfg.attrs = attr;
  cfg.numAttrs = na;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return e;
  }
  return cudaGetLastError();
}

}  // namespace arn
