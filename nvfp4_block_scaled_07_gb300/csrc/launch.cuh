// Host-side kernel launch with programmatic dependent launch (PDL).
//
// A kernel of the library starts with griddepcontrol.wait before it touches
// global memory, and signals griddepcontrol.launch_dependents only after, so a
// kernel launched here behind another kernel may be scheduled while its
// predecessor drains; its reads and writes still happen after the predecessor
// has completed.  Because the signal comes after the wait, a kernel that runs
// early finds everything before its predecessor complete.  stream_kernel
// (few_stream.cu), always launched behind a kernel of the same call, rests on
// that: its producer warps read the call's weights, ids and plan, which that
// predecessor does not write (of the gated product: the ids, not the plan),
// before the wait.  A kernel that signals before its own wait must not be
// followed by one that does so.  NVFP4MOE_PDL=0 in the environment launches
// without the attribute (plain stream order), for comparisons.
#pragma once

#include <cstdlib>
#include <utility>

#include <cuda_runtime.h>

namespace nvfp4moe {

inline bool pdl_enabled() {
  static const bool on = [] {
    const char* v = std::getenv("NVFP4MOE_PDL");
    return !(v && v[0] == '0');
  }();
  return on;
}

template <typename... KArgs, typename... Args>
cudaError_t launch_kernel(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                          bool cooperative, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  if (cooperative) {
    // A grid whose CTAs wait on one another: all of them resident at once.
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
  } else {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  }
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

}  // namespace nvfp4moe
