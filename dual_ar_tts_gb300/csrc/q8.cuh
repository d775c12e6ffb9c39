// Launches of the 8-bit operators.
//
// Each may be scheduled before the kernel in front of it on its stream has ended (programmatic stream serialisation) and waits
// for that on the device, before it reads or writes anything but its own shared memory: a run of these short kernels does
// not pay a launch's latency each time (7 rows of 6144 x 2560 7.7 -> 6.8 us, one row's norm 2.8 -> 2.4).  What the kernel in
// front may have written is not read through the read-only path: it was not constant while this kernel ran.
#pragma once

#include <cuda_runtime.h>

#include <type_traits>

#include "../../include/s2frame.h"

namespace s2 {

template <typename... Args>
inline int launch_ahead(void (*kernel)(Args...), dim3 grid, dim3 cluster, int threads, int smem, cudaStream_t st,
                        const std::decay_t<Args>&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster.x;
  at[1].val.clusterDim.y = cluster.y;
  at[1].val.clusterDim.z = cluster.z;
  cfg.attrs = at;
  cfg.numAttrs = cluster.x * cluster.y * cluster.z > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? S2_OK : S2_ECUDA;
}

}  // namespace s2
