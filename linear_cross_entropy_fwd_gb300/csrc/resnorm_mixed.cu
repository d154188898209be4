// resnorm_mixed.cu -- the residual join's kernels: bf16 y and z on an fp32 stream.
#include "resnorm_bwd.cuh"
#include "resnorm_fwd.cuh"

namespace flce {
cudaError_t launch_resnorm_fwd_mixed(const NormParams& p, int sms, cudaStream_t s) {
  return launch_fwd_types<bf16_t, float>(p, sms, s);
}
cudaError_t launch_resnorm_bwd_mixed(NormParams& p, int64_t parts, cudaStream_t s) {
  return launch_bwd_types<bf16_t, float>(p, parts, s);
}
}  // namespace flce
