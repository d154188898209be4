// resnorm_bwd_bf16.cu -- the residual join's backward kernels: bf16 y and z on a bf16 stream.
#include "resnorm_bwd.cuh"

namespace flce {
cudaError_t launch_resnorm_bwd_bf16(const NormParams& p, int64_t parts, cudaStream_t s) {
  return launch_bwd_types<bf16_t, bf16_t>(p, parts, s);
}
}  // namespace flce
