// slm_norm_bf16.cu - the block norm's kernels for bf16 rows (one source per type: they compile side
// by side).
#include "slm_norm.cuh"

namespace slm {
cudaError_t norm_fwd_bf16(const NormFwd& p, cudaStream_t s) { return fwd_t<__nv_bfloat16>(p, s); }
cudaError_t norm_bwd_bf16(const NormBwd& p, const DevCtl& c, cudaStream_t s) {
  return bwd_t<__nv_bfloat16>(p, c, s);
}
cudaError_t norm_ran_out_bf16(int* flags) { return take_ran_out(flags); }
}  // namespace slm
