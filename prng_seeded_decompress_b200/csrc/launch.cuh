// launch.cuh -- launching kernels with programmatic dependent launch: the
// kernel may start while the one before it on the stream is finishing, and
// calls grid_wait() before it reads or writes anything that kernel touches.  What
// that kernel may write is not constant for the life of this one: it is read with
// plain loads, not through the read-only path (__ldg, or a kernel's own const
// __restrict__ pointers), which the compiler may also move above the wait.
#pragma once

#include <cuda_runtime.h>

#include <utility>

#include "between_internal.h"

namespace seedlm {

// Returns once every grid before this one on the stream has completed and
// its writes are visible.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Lets the next grid on the stream start once every CTA of this one has called
// this or ended.
__device__ __forceinline__ void grid_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <class... Params, class... Args>
int launch_pdl_cluster(void (*kernel)(Params...), dim3 grid, dim3 threads, size_t smem, int cluster, cudaStream_t stream,
                       Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = threads;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t err = cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
  if (err != cudaSuccess) {
    cudaGetLastError();  // the caller has the error; the next call starts clean
    return record_cuda_error(err);
  }
  count_launch();
  return SEEDLM_OK;
}

template <class... Params, class... Args>
int launch_pdl(void (*kernel)(Params...), dim3 grid, dim3 threads, size_t smem, cudaStream_t stream, Args&&... args) {
  return launch_pdl_cluster(kernel, grid, threads, smem, 1, stream, std::forward<Args>(args)...);
}

}  // namespace seedlm
