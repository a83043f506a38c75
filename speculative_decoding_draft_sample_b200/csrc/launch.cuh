// Launches that set themselves up while the launch before them in the stream still
// runs, and the device side of that.
//
// kAfter: reads what it likes; it waits (grid_wait) for the launch before to be complete
// ahead of its first access to global memory, its own barriers and tensor memory set up.
// In a stream of such calls each takes 2 us less (norm of m1536 h7168 to e4m3 18.5 ->
// 16.2 us, a product of m1 n4096 k4096 12.9 -> 10.2).
// kBeside: shares no output with the launch before and no input that either writes;
// it works at once and waits before it ends.
// Either way a launch is complete only after the one before it. grid_release lets the
// next launch's CTAs start on SMs that come free; without it they start at the kernel's
// end. A kernel that a kBeside launch follows, which relies on all that the kernel itself
// relies on, releases after its own grid_wait. The products release (m1536 n129280 k4096
// e4m3 573 us in short runs, 584 without), so do kernels that a launch of the same call follows; norm
// and log probabilities do not (16.5 and 44 us, 16.2 and 40 without, for m1536 h7168 and
// b64 j6 v151936 fp32: early CTAs of the next call leave this one's rows uneven).
#pragma once

#include <cuda_runtime.h>

namespace dspark {

enum Order : int { kAfter, kBeside };

__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// cluster: CTAs of a cluster (1: none)
template <typename... P, typename... Args>
cudaError_t launch_early(void (*kern)(P...), dim3 blocks, int threads, int smem, int cluster, cudaStream_t s, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = blocks;
  cfg.blockDim = dim3(threads);
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
  return cudaLaunchKernelEx(&cfg, kern, P(args)...);
}

}  // namespace dspark
