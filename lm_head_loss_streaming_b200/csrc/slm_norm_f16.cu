// slm_norm_f16.cu - the block norm's kernels for fp16 rows (one source per type: they compile side
// by side).
#include "slm_norm.cuh"

namespace slm {
cudaError_t norm_fwd_f16(const NormFwd& p, cudaStream_t s) { return fwd_t<__half>(p, s); }
cudaError_t norm_bwd_f16(const NormBwd& p, const DevCtl& c, cudaStream_t s) {
  return bwd_t<__half>(p, c, s);
}
cudaError_t norm_ran_out_f16(int* flags) { return take_ran_out(flags); }
}  // namespace slm
