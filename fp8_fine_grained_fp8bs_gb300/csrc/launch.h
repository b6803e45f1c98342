// Launch helper of the small kernels that run one behind the other.
#pragma once

#include <cuda_runtime.h>

namespace fp8bs {

// Launches with programmatic stream serialisation: the kernel may be set up
// while the one before it on the stream ends.  Every thread of it has to call
// griddep_wait() before it touches memory.
template <typename... P, typename... A>
cudaError_t launch_behind_smem(void (*kern)(P...), dim3 grid, unsigned threads, size_t smem_bytes, cudaStream_t stream,
                               const A&... args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem_bytes;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename... P, typename... A>
cudaError_t launch_behind(void (*kern)(P...), dim3 grid, unsigned threads, cudaStream_t stream, const A&... args) {
  return launch_behind_smem(kern, grid, threads, 0, stream, args...);
}

}  // namespace fp8bs
