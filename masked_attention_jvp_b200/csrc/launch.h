// Launches of the block operators' kernels with programmatic stream serialization: the
// kernel may start while the one before it on the stream drains, and waits for it on the
// device (begin_after_previous) before it touches global memory. Short calls in a row save
// most of the gap between two kernels, about 1 us.
#pragma once
#include <cuda_runtime.h>

namespace caj {

#ifdef __CUDACC__
// First statement of such a kernel (after set-up that touches no global memory): everything
// that earlier kernels of the stream wrote is visible after it. Then lets the next one start.
__device__ __forceinline__ void begin_after_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
#endif

template <typename... Params, typename... Args>
cudaError_t launch_in_order(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                            const Args &...args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, Params(args)...);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace caj
