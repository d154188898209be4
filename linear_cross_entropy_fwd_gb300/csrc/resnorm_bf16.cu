// resnorm_bf16.cu -- the residual join's kernels: bf16 y and z on a bf16 stream.
#include "resnorm_bwd.cuh"
#include "resnorm_fwd.cuh"

namespace flce {
cudaError_t launch_resnorm_fwd_bf16(const NormParams& p, int sms, cudaStream_t s) {
  return launch_fwd_types<bf16_t, bf16_t>(p, sms, s);
}
cudaError_t launch_resnorm_bwd_bf16(NormParams& p, int64_t parts, cudaStream_t s) {
  return launch_bwd_types<bf16_t, bf16_t>(p, parts, s);
}
}  // namespace flce
