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

// For a kernel that reads nothing of the one before it on the stream, only what was there
// before that one (which began by begin_after_previous, so all of it is in place): in place of
// begin_after_previous, last in one block. The grid then ends after its predecessor's end,
// which is what the next kernel's wait relies on.
#ifdef __CUDACC__
__device__ __forceinline__ void end_after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
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
