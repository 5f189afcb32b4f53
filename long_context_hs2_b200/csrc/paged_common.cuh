// Device helpers of the paged decode path's kernels.
#pragma once

#include "tc_common.cuh"

namespace hs2 {

// Registers moved between the warpgroups of a block: a warpgroup gives up what it
// has above N, or takes up to N from what others gave up.  All shares together
// must not pass what the block was launched with.
template <int N>
__device__ __forceinline__ void regs_give_up() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_take() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// 1 / x to within an ulp or so (normal x).
__device__ __forceinline__ float fast_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

}  // namespace hs2
