// slm_ran_out.cuh - a word per device and source file that remembers waits which ran out, for the
// operators whose callers usually drop the workspace that holds a call's status word.
#pragma once

#include "slm_internal.h"

namespace slm {
namespace {

__device__ int g_ran_out;

// By one thread of a block whose wait ran out, as the block ends.
__device__ __forceinline__ void record_ran_out() { atomicOr(&g_ran_out, kFlagTimeout); }

// Adds the current device's word to *flags and clears it.  Synchronises.
inline cudaError_t take_ran_out(int* flags) {
  int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_ran_out, sizeof(int));
  if (e != cudaSuccess || v == 0) return e;
  *flags |= v;
  v = 0;
  return cudaMemcpyToSymbol(g_ran_out, &v, sizeof(int));
}

}  // namespace
}  // namespace slm
