// resnorm_bwd_fp32.cu -- the residual join's backward kernels: fp32 throughout.
#include "resnorm_bwd.cuh"

namespace flce {
cudaError_t launch_resnorm_bwd_fp32(const NormParams& p, int64_t parts, cudaStream_t s) {
  return launch_bwd_types<float, float>(p, parts, s);
}
}  // namespace flce
