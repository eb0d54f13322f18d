// Launches that overlap their set-up with the work before them on the stream.
#pragma once

#include <cuda_runtime.h>

namespace pa {

// A launch as a programmatic dependent of the work before it on the stream: it may be set up during
// that work's tail, and its kernel starts with await_previous(), before any access to memory. Measured
// against plain launches, calls in a row: 31 rotary rows 4.1 -> 3.1 us, 4,127 17.3 -> 15.1, a plan of
// 32 requests 8.2 -> 5.4, one of 4,096 10.3 -> 8.8. (These kernels letting the next one be
// set up early in turn gained nothing more.)
template <class... Params, class... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), dim3 grid, unsigned block, size_t smem,
                             cudaStream_t stream, int cluster, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 0 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

__device__ __forceinline__ void await_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Lets the next dependent launch of the stream be set up while this kernel still runs (it waits in its
// await_previous() all the same). For the first of a call's two short launches: without and with it, a selection of one
// request 7.9 and 7.6 us, a fork of four rows 13.5 and 13.2. (The shared decode's attention, all of whose shared memory
// and threads are in use, is slower with it: four rows 13.4 and 14.2.)
__device__ __forceinline__ void launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

}  // namespace pa
