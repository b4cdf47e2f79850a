// Device and launch helpers of the training operators' kernels.
#pragma once

#include <cuda_bf16.h>

#include "xp_train_internal.h"

namespace xp {

// Every kernel of the training operators may start while its predecessor in
// the stream drains (programmatic dependent launch) and calls this before it
// touches anything another kernel may write: it waits until all earlier
// kernels are done and their writes visible.  A CTA that ends without it
// would let the successor overtake the predecessor, so every thread calls it.
__device__ __forceinline__ void wait_for_predecessors() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The successor's CTAs may be placed from now on, as this grid's make room.
__device__ __forceinline__ void let_successor_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// What every kernel that takes more than the default may take: the attribute is
// the function's, not a launch's, so it has one value whoever sets it.  (Set to
// each call's own size, a thread's call lowered it under another's larger one.)
constexpr size_t kMaxDynamicSmem = 224 * 1024;
constexpr size_t kMaxStaticSmem = 3 * 1024;   // beside it, of the 227 KiB a CTA may have
template <typename... Params>
cudaError_t allow_dynamic_smem(void (*kernel)(Params...)) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxDynamicSmem);
}

// One launch, with programmatic dependence on the work before it (a stream of
// small steps: 8.3 us each without, 4.0 with it); csize > 1: in clusters of
// that many CTAs, and without it, as clusters placed beside a kernel that
// drains held each other up (layer norm backward 2000 x 40032: 169 us with it,
// 116 without).
template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), dim3 grid, int block, size_t smem, int csize, cudaStream_t st,
                             Args... args) {
  if (smem > 40 * 1024) {   // with what the kernel takes statically, more than the 48 KiB every kernel may have
    const cudaError_t e = allow_dynamic_smem(kernel);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = csize;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = csize > 1 ? at + 1 : at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, Params(args)...);
}

}  // namespace xp
