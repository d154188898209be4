// host_util.h -- host services of libflce that every entry point's source
// file shares: the error text, device checks, scratch, and the status word
// (internal; implemented in flce_api.cu and step_common.cu).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

#include "../../include/flce.h"
#include "flce_internal.h"

namespace flce {

// Further bits of the per-call device status word (see flce_internal.h).
enum : int32_t {
  FLCE_DEV_SEQLENS = 4,  // sequence offsets out of order or outside [0, T]
};

void host_clear_error();
int host_error(int status, const char* fmt, ...);  // sets the text, returns `status`
int host_cuda_error(cudaError_t e, const char* what);
int host_device(int* sms);  // the current device's SM count; FLCE_ERR_ARCH if not 10.3
int host_pool_alloc(void** p, size_t bytes, cudaStream_t s);
int host_status(int32_t bits);  // status word -> flce_status, with its text

// A tiled tensor map of `rank` dimensions (dim 0 contiguous, 128-byte swizzle,
// zero fill outside); `pitch` holds the byte strides of dims 1 .. rank-1.
int host_tensor_map(CUtensorMap* m, const void* base, CUtensorMapDataType dt, int rank,
                    const uint64_t* dims, const uint64_t* pitch, const uint32_t* box,
                    const char* what);

#define FLCE_TRY(call)                                                 \
  do {                                                                 \
    const cudaError_t e_ = (call);                                     \
    if (e_ != cudaSuccess) return ::flce::host_cuda_error(e_, #call);  \
  } while (0)

// A kernel's dynamic shared-memory limit, raised once per device (that costs
// about as much as a launch).
class SmemLimit {
 public:
  template <class KernelT>
  cudaError_t raise(KernelT kernel, size_t bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = uint64_t{1} << (dev & 63);
    if (done_.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(bytes));
    if (e == cudaSuccess) done_.fetch_or(bit, std::memory_order_release);
    return e;
  }

 private:
  std::atomic<uint64_t> done_{0};  // devices 0 .. 63 (host_device refuses others)
};

inline size_t round256(size_t x) { return (x + 255) / 256 * 256; }

// One call of an operator: its scratch (the caller's, or the library's
// stream-ordered pool), the status word at its start, and the reporting of
// that word after the last launch.
struct StepCall {
  cudaStream_t stream = nullptr;
  uint8_t* scratch = nullptr;   // `bytes` bytes after the status word
  int32_t* status = nullptr;    // device status word; nullptr when nothing needs it
  // kIfAsked: a status word only if the caller looks at it; kCleared: always;
  // kKernelClears: always, and the call's first kernel writes it.
  enum Status { kIfAsked, kCleared, kKernelClears };
  int begin(const flce_opts& o, size_t bytes, Status mode);
  int end(int rc);              // rc: what the launches returned

 private:
  const flce_opts* o_ = nullptr;
  uint8_t* base_ = nullptr;
  bool owned_ = false;
};

// The options of a call: a copy of the caller's, or the defaults.
inline flce_opts opts_or_default(const flce_opts* in) {
  flce_opts o;
  flce_opts_init(&o);
  if (in) o = *in;
  return o;
}

// A 16-byte aligned address.
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace flce
