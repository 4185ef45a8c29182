// call_common.h -- overlap checks, overlapped launches and the stall control, for the calls
// on norms and pools (k_norm_rope.cu, pool_share.cu, pool_prefill.cu, k_prefill_pool_tc.cu).
#pragma once

#include "duo_internal.h"

namespace duo {

// Is the test control duo_debug_device_stall on?
bool device_stall();

// A byte range of a call's tensors, for its overlap check.
struct Span {
  uintptr_t lo, hi;
  bool meets(const Span &o) const { return lo < o.hi && o.lo < hi; }
};

// A launch whose start may overlap the end of the kernel before it in the stream: the
// kernel executes griddepcontrol.wait before it reads or writes global memory.
template <class Param>
cudaError_t launch_overlapped(void (*kernel)(Param), int64_t blocks, int threads, int smem, cudaStream_t st,
                              const Param &param) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, param);
}

}  // namespace duo
