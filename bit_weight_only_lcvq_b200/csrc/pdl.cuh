// Launch with programmatic dependent launch: the kernel may become resident while
// the one before it on the stream finishes.  Only for kernels that call
// griddepcontrol.wait before they touch memory, trigger their own dependents only
// after it, and read what earlier kernels wrote with ordinary loads (see common.cuh).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace lcvq {

template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kern)(KArgs...), int64_t grid, int threads, size_t smem, cudaStream_t s,
                       const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaError_t e = cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...); e != cudaSuccess)
    return e;
  return cudaGetLastError();
}

}  // namespace lcvq
