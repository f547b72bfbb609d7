// Launches whose set-up overlaps the end of the work before them on their
// stream (programmatic dependent launch).
//
// Kernels launched so call grid_dependency_wait() in every thread before they
// touch global memory: it returns once all earlier work on the stream has
// completed and its writes are visible.  A kernel may call
// grid_dependents_launch() as soon as it likes: a following launch of this
// kind then takes free SM resources, sets up and waits.  Any other kernel
// before or after is ordered as always.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace bwg {

__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_dependents_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Reads of what the work before may have written.  Not ld.global.nc (__ldg, const
// __restrict__): that is for memory that nobody writes while the kernel runs, and
// here it starts earlier.  Volatile loads stay behind the wait; the one of 16
// bytes may move past stores, which never go to an input, but takes its pointer
// out of behind_wait() (C++ loads, which keep to the order of the stores, take the
// combine's gradient of 4096 x 8, H = 4096 BF16 from 86.5 us to 98.7).
template <class T>
__device__ __forceinline__ T* behind_wait(T* p) {
  asm volatile("" : "+l"(p)::"memory");
  return p;
}
__device__ __forceinline__ uint4 ld_global(const uint4* p) {
  uint4 v;
  asm("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t ld_global(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ uint16_t ld_global(const uint16_t* p) {
  uint16_t v;
  asm volatile("ld.global.b16 %0, [%1];" : "=h"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ float ld_global(const float* p) {
  float v;
  asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}
// The same for what this SM reads once: the narrow ones leave no line in L1.
__device__ __forceinline__ uint4 ld_global_once(const uint4* p) { return ld_global(p); }
__device__ __forceinline__ uint32_t ld_global_once(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.global.L1::no_allocate.b32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ uint16_t ld_global_once(const uint16_t* p) {
  uint16_t v;
  asm volatile("ld.global.L1::no_allocate.b16 %0, [%1];" : "=h"(v) : "l"(p));
  return v;
}

// Launch of a grid of clusters whose kernel waits so, for kernels that take their
// parameters as one block.
template <class P>
cudaError_t launch_behind(void (*kernel)(P), unsigned grid, unsigned threads, size_t smem, cudaStream_t s,
                          unsigned cluster, const P& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <class... Params, class... Args>
cudaError_t launch_overlapped(void (*kernel)(Params...), unsigned grid, unsigned threads, size_t smem, cudaStream_t s,
                              unsigned cluster, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Args&&>(args)...);
}

}  // namespace bwg
