// Launches that overlap their start with the end of the kernel ahead of them on
// the stream (programmatic dependent launch).
//
// A kernel launched with launch_early may be resident before the kernel ahead has
// ended. It calls pdl_wait() in every thread before it reads or writes global
// memory and before it returns: the wait ends when the kernel ahead has completed
// and its writes are visible, and so, because that kernel waited too, everything
// before it. pdl_launch() lets the kernel behind take its place early.
// Such a kernel reads with plain loads (or TMA) only: the read-only path (__ldg) is
// for memory that does not change from a kernel's start on, and its start comes
// before the writes of the kernel ahead.
#pragma once

#include <cuda_runtime.h>

#include "tm.h"

namespace trimix {

__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// cluster: thread blocks of a cluster along x (1: none).
template <class... P, class... A>
int launch_early(void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t st, int cluster,
                 const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess) return TM_OK;
  cudaGetLastError();
  return TM_ERR_CUDA;
}

}  // namespace trimix
