// resnorm_fp32.cu -- the residual join's kernels: fp32 throughout.
#include "resnorm_bwd.cuh"
#include "resnorm_fwd.cuh"

namespace flce {
cudaError_t launch_resnorm_fwd_fp32(const NormParams& p, int sms, cudaStream_t s) {
  return launch_fwd_types<float, float>(p, sms, s);
}
cudaError_t launch_resnorm_bwd_fp32(NormParams& p, int64_t parts, cudaStream_t s) {
  return launch_bwd_types<float, float>(p, parts, s);
}
}  // namespace flce
