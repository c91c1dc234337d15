// Programmatic dependent launch: a kernel of these operators may be set up
// while the one before it on the stream still runs.  It waits for that one's
// end, and so for all before it, ahead of its first access to memory
// (follow_previous), and lets the next one do the same (allow_next).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace fp8q {

__device__ __forceinline__ void follow_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void allow_next() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Launch configuration with the attribute, and clusters of `cluster` CTAs.
struct Launch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  Launch(unsigned grid_x, unsigned grid_y, int threads, size_t smem, cudaStream_t stream,
         int cluster = 1) {
    cfg.gridDim = dim3(grid_x, grid_y, 1);
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
  }
  Launch(const Launch &) = delete;
  template <typename... P, typename... A>
  cudaError_t run(void (*kernel)(P...), A &&...args) {
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<A &&>(args)...);
  }
};

}  // namespace fp8q
