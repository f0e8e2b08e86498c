// Launches that overlap the end of the kernel before them.
#pragma once
#include <cuda_runtime.h>

#include "../../include/attn_slice.h"

namespace attn {

// Waits until the grids before this one on the stream have ended and their
// memory is visible: to ordinary loads, not to those of the read-only path
// (ld.global.nc), which may give what the SM read before.  So whatever an earlier
// call may have written (lengths, tables, lists, queries) is read by ordinary ones.
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Lets the next grid on the stream start where it asks to start early.
__device__ __forceinline__ void admit_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename K>
inline int raise_smem(K kern, size_t bytes, bool *done) {
  if (*done) return ATTN_OK;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes)) != cudaSuccess)
    return ATTN_ERR_CUDA;
  *done = true;
  return ATTN_OK;
}

// A launch that may start while the one before it on the stream drains: its
// prologue hides the latency of the launch.  Each such kernel, every block of
// it, calls after_previous() before it touches memory (or, where it is told
// that it depends on nothing of the kernel before it, ahead of its end), so the
// end of one grid on the stream still implies the end of those before it.
template <typename... A>
inline int launch_after(void (*kern)(A...), dim3 grid, int threads, size_t smem, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

constexpr size_t kSmemMax = 232448;

}  // namespace attn
