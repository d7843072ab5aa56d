// launch_after.cuh — launches chained by programmatic stream serialization.
#pragma once

#include <cuda_runtime.h>

namespace tgdn {

// A launch that may be scheduled while the kernel before it in the stream drains (it waits
// for that kernel's completion before it reads anything).
template <typename... P, typename... A>
static cudaError_t launch_after(void (*kern)(P...), dim3 grid, dim3 block, size_t smem,
                                cudaStream_t s, const A&... args) {
  cudaLaunchConfig_t lc = {};
  lc.gridDim = grid;
  lc.blockDim = block;
  lc.dynamicSmemBytes = smem;
  lc.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&lc, kern, args...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace tgdn
