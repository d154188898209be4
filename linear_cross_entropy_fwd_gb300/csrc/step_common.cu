// step_common.cu -- scratch and status reporting shared by the operators that
// stand around the head (embedding, packed attention, orthogonalisation).
#include "host_util.h"

namespace flce {
namespace {

__global__ void step_status_kernel(const int32_t* bits, int32_t* out) {
  const int32_t b = *bits;
  *out = (b & FLCE_DEV_TIMEOUT)   ? FLCE_ERR_TIMEOUT
         : (b & FLCE_DEV_TARGET)  ? FLCE_ERR_TARGET
         : (b & FLCE_DEV_SEQLENS) ? FLCE_ERR_ARG
                                  : FLCE_OK;
}

constexpr size_t kStatusBytes = 256;

}  // namespace

int StepCall::begin(const flce_opts& o, size_t bytes, Status mode) {
  o_ = &o;
  stream = static_cast<cudaStream_t>(o.stream);
  const bool want = mode != kIfAsked || o.status_dev || o.sync;
  const size_t total = (want ? kStatusBytes : 0) + bytes;
  if (o.workspace_used) *o.workspace_used = kStatusBytes + bytes;
  if (total == 0) return FLCE_OK;
  if (o.workspace) {
    if (o.workspace_bytes < kStatusBytes + bytes)
      return host_error(FLCE_ERR_WORKSPACE,
                        "workspace of %zu bytes is smaller than the %zu bytes this call needs",
                        o.workspace_bytes, kStatusBytes + bytes);
    if (reinterpret_cast<uintptr_t>(o.workspace) & 255u)
      return host_error(FLCE_ERR_ALIGN, "workspace must be 256-byte aligned");
    base_ = static_cast<uint8_t*>(o.workspace);
  } else {
    void* p = nullptr;
    const int rc = host_pool_alloc(&p, total, stream);
    if (rc) return rc;
    base_ = static_cast<uint8_t*>(p);
    owned_ = true;
  }
  scratch = base_ + (want ? kStatusBytes : 0);
  if (want) {
    status = reinterpret_cast<int32_t*>(base_);
    const cudaError_t e = mode == kKernelClears
                              ? cudaSuccess
                              : cudaMemsetAsync(status, 0, sizeof(int32_t), stream);
    if (e != cudaSuccess) return end(host_cuda_error(e, "cudaMemsetAsync(status)"));
  }
  return FLCE_OK;
}

int StepCall::end(int rc) {
  int32_t bits = 0;
  if (rc == FLCE_OK && o_->status_dev) {
    step_status_kernel<<<1, 1, 0, stream>>>(status, o_->status_dev);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) rc = host_cuda_error(e, "status");
  }
  if (rc == FLCE_OK && o_->sync) {
    const cudaError_t e =
        cudaMemcpyAsync(&bits, status, sizeof bits, cudaMemcpyDeviceToHost, stream);
    if (e != cudaSuccess) rc = host_cuda_error(e, "cudaMemcpyAsync(status)");
  }
  if (owned_) {
    owned_ = false;
    const cudaError_t e = cudaFreeAsync(base_, stream);
    if (e != cudaSuccess && rc == FLCE_OK) rc = host_cuda_error(e, "cudaFreeAsync(workspace)");
  }
  if (rc == FLCE_OK && o_->sync) {
    const cudaError_t e = cudaStreamSynchronize(stream);
    if (e != cudaSuccess) return host_cuda_error(e, "cudaStreamSynchronize");
    rc = host_status(bits);
  }
  return rc;
}

}  // namespace flce
