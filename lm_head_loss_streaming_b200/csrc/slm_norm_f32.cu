// slm_norm_f32.cu - the block norm's kernels for fp32 rows (one source per type: they compile side
// by side).
#include "slm_norm.cuh"

namespace slm {
cudaError_t norm_fwd_f32(const NormFwd& p, cudaStream_t s) { return fwd_t<float>(p, s); }
cudaError_t norm_bwd_f32(const NormBwd& p, const DevCtl& c, cudaStream_t s) {
  return bwd_t<float>(p, c, s);
}
cudaError_t norm_ran_out_f32(int* flags) { return take_ran_out(flags); }
}  // namespace slm
