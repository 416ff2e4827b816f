// slm_wait.cuh - the bounded pipeline wait shared by the GEMM kernels and the block norm's ring.
#pragma once

#include "slm_internal.h"
#include "sm100.cuh"

namespace slm {

// Bounded wait executed by all 32 lanes of a warp; the result is warp-uniform.
// honor_abort = false is used for the final waits on a CTA's own in-flight work.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort,
                                          const DevCtl& ctl, bool honor_abort = true) {
  const uint32_t a = sm100::smem_u32(bar);
  bool done = sm100::mbar_try_wait(a, parity);
  if (!done) {
    const long long t0 = clock64();
    while (true) {
      done = sm100::mbar_try_wait(a, parity);
      if (done) break;
      if (honor_abort && *abort) break;
      if (clock64() - t0 > ctl.timeout_cycles) {
        *abort = 1;
        atomicOr(ctl.status, kFlagTimeout);
        break;
      }
    }
  }
  return __all_sync(0xffffffffu, done);
}

}  // namespace slm
