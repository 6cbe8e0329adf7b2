// Launches that follow one another closely: each may start while the one ahead of it still runs, sets up what it
// needs, and waits for the other's end (grid_wait) before it touches memory; grid_launch_dependents lets the next one
// start.  Every kernel waits before it lets the next one start, so that the end of a launch means the end of all
// launches ahead of it.
#ifndef E4B_LAUNCH_CUH
#define E4B_LAUNCH_CUH

#include <cuda_runtime.h>

namespace e4b {

__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// S > 0: in clusters of S blocks.
template <typename... Params, typename... Args>
cudaError_t launch_following(void (*kernel)(Params...), int grid, int threads, int smem, int S, cudaStream_t stream,
                             const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)S;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = S > 0 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace e4b

#endif  // E4B_LAUNCH_CUH
