// slm_norm.cu - the block norm's row plan and its dispatch by type (kernels: slm_norm.cuh).
#include <algorithm>

#include "slm_internal.h"

namespace slm {

cudaError_t norm_fwd_bf16(const NormFwd& p, cudaStream_t s);
cudaError_t norm_fwd_f16(const NormFwd& p, cudaStream_t s);
cudaError_t norm_fwd_f32(const NormFwd& p, cudaStream_t s);
cudaError_t norm_bwd_bf16(const NormBwd& p, const DevCtl& c, cudaStream_t s);
cudaError_t norm_bwd_f16(const NormBwd& p, const DevCtl& c, cudaStream_t s);
cudaError_t norm_bwd_f32(const NormBwd& p, const DevCtl& c, cudaStream_t s);
cudaError_t norm_ran_out_bf16(int* flags);
cudaError_t norm_ran_out_f16(int* flags);
cudaError_t norm_ran_out_f32(int* flags);

NormPlan norm_plan(int64_t N, int64_t rows_per_gate, bool has_gate, int max_blocks, int batch,
                   int classes) {
  NormPlan q{};
  q.shared_gate = has_gate && rows_per_gate > 1;
  q.rows = q.shared_gate ? rows_per_gate : N;
  q.groups = q.shared_gate ? N / rows_per_gate : 1;
  q.classes = classes;
  // Blocks own either one part (a slice's rows of one class) of one group or several whole
  // groups.
  const int64_t most = (q.rows + batch * classes - 1) / (batch * classes);  // a batch of rows each
  q.slices = static_cast<int>(
      std::max<int64_t>(1, std::min<int64_t>(most, max_blocks / (q.groups * classes))));
  q.blocks = static_cast<int>(q.parts() > 1 ? q.groups * q.parts()
                                            : std::min<int64_t>(q.groups, max_blocks));
  return q;
}

cudaError_t launch_norm_fwd(int dtype, const NormFwd& p, cudaStream_t s) {
  return dtype == 0 ? norm_fwd_bf16(p, s) : dtype == 1 ? norm_fwd_f16(p, s) : norm_fwd_f32(p, s);
}

cudaError_t launch_norm_bwd(int dtype, const NormBwd& p, const DevCtl& c, cudaStream_t s) {
  return dtype == 0   ? norm_bwd_bf16(p, c, s)
         : dtype == 1 ? norm_bwd_f16(p, c, s)
                      : norm_bwd_f32(p, c, s);
}

cudaError_t norm_ran_out(int* flags) {
  cudaError_t e = norm_ran_out_bf16(flags);
  if (e == cudaSuccess) e = norm_ran_out_f16(flags);
  return e == cudaSuccess ? norm_ran_out_f32(flags) : e;
}

}  // namespace slm
