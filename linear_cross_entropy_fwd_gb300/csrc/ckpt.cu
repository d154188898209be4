// ckpt.cu -- storing activations in 8 bits and reading them back (ckpt.cuh has the format).
//
// Bound by memory: 2 or 4 bytes a value on one side, 8.25 bits on the other.  A thread holds
// an octet, four neighbouring lanes a group that shares a scale.  65536 x 4096 in bf16: saved in
// 126 us (6.5 TB/s), loaded in 117 (7.0 TB/s); 32768 x 4096 in fp32 95 and 100 us (an octet
// stored in halves: 126).
#include "ckpt.cuh"
#include "host_util.h"

namespace flce {
namespace {

constexpr int kThreads = 256, kOctets = 4;  // octets of a thread, loaded together

struct CkptParams {
  Ckpt c;
  void* x;
  int64_t x_row;
  uint32_t octets;  // of a row of x
  uint32_t padded;  // of a row of codes, its padding included (save), or of x (load)
  int64_t total;    // of all rows, `padded` each
  int32_t* clear;
  bool wide;        // x is 32-byte aligned
};

// A thread's octets, kThreads apart: row and octet of each.  One 64-bit division for a CTA,
// one of 32 bits for a thread, and for rows longer than a step none after it.
struct Place {
  int64_t row;
  uint32_t o;
  __device__ __forceinline__ Place(int64_t cta, uint32_t padded) {
    row = cta / padded;
    o = static_cast<uint32_t>(cta - row * padded) + threadIdx.x;
    wrap(padded);
  }
  __device__ __forceinline__ void wrap(uint32_t padded) {
    const uint32_t q = o / padded;
    row += q;
    o -= q * padded;
  }
  __device__ __forceinline__ void next(uint32_t padded) {
    o += kThreads;
    if (padded < kThreads) {
      wrap(padded);
    } else if (o >= padded) {
      o -= padded;
      ++row;
    }
  }
};

template <class T>
__global__ void __launch_bounds__(kThreads) ckpt_save_kernel(const CkptParams p) {
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kThreads * kOctets);
  Place at(first, p.padded);
  typename Elem<T>::Octet v[kOctets];
  uint8_t* scales[kOctets];
  int o[kOctets];
#pragma unroll
  for (int k = 0; k < kOctets; ++k) {
    const bool there = first + threadIdx.x + k * kThreads < p.total;
    o[k] = there ? at.o : p.padded;  // `padded` stores nothing
    scales[k] = p.c.scales + at.row * p.c.spitch;
    v[k] = {};
    if (there && at.o < p.octets)
      v[k] = *(static_cast<const typename Elem<T>::Octet*>(row_at<T>(p.x, at.row, p.x_row)) + at.o);
    at.next(p.padded);
  }
  // the codes of all rows follow one another
  uint8_t* codes = p.c.codes + (first + threadIdx.x) * 8;
#pragma unroll
  for (int k = 0; k < kOctets; ++k)
    ckpt_store_octet(p.c, codes + k * kThreads * 8, scales[k], o[k], v[k]);
}

// With `clear`, which becomes 0, the next launch knows that it may start meanwhile; other
// callers' may be anything.
template <class T>
__global__ void __launch_bounds__(kThreads) ckpt_load_kernel(const CkptParams p) {
  if (p.clear) {
    grid_launch_dependents();
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.clear = 0;
  }
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kThreads * kOctets);
  Place at(first, p.padded);
  uint2 codes[kOctets];
  uint32_t scale[kOctets];
  typename Elem<T>::Octet* to[kOctets];
#pragma unroll
  for (int k = 0; k < kOctets; ++k) {
    to[k] = nullptr;
    if (first + threadIdx.x + k * kThreads < p.total) {
      to[k] = static_cast<typename Elem<T>::Octet*>(row_at<T>(p.x, at.row, p.x_row)) + at.o;
      codes[k] = *reinterpret_cast<const uint2*>(p.c.codes + at.row * p.c.pitch + at.o * 8);
      scale[k] = p.c.scales[at.row * p.c.spitch + (at.o >> 2)];
    }
    at.next(p.padded);
  }
#pragma unroll
  for (int k = 0; k < kOctets; ++k)
    if (to[k]) put_octet(to[k], to_octet(T{}, ckpt_octet(codes[k], scale[k])), p.wide);
}

CkptParams params(const Ckpt& c, void* x, int64_t x_row, int64_t N, int64_t H, bool save) {
  CkptParams p{};
  p.c = c;
  p.x = x;
  p.x_row = N > 1 ? x_row : H;
  p.octets = static_cast<uint32_t>(H / 8);
  p.padded = save ? static_cast<uint32_t>(p.c.pitch) / 8 : p.octets;
  p.total = N * p.padded;
  p.wide = (reinterpret_cast<uintptr_t>(x) & 31) == 0;
  return p;
}

unsigned grid_of(const CkptParams& p) {
  return static_cast<unsigned>((p.total + kThreads * kOctets - 1) / (kThreads * kOctets));
}

int check(const char* fn, const void* x, int64_t x_row, int64_t N, int64_t H, const void* ckpt,
          int32_t dtype) {
  if (dtype != FLCE_BF16 && dtype != FLCE_FP32)
    return host_error(FLCE_ERR_ARG, "%s: unknown dtype %d", fn, dtype);
  if (N < 0 || N >= (int64_t{1} << 31) || H < 1 || H > (int64_t{1} << 20))
    return host_error(FLCE_ERR_ARG, "%s: sizes must satisfy 0 <= N < 2^31, 1 <= H <= 2^20", fn);
  if (H % 8 != 0) return host_error(FLCE_ERR_ALIGN, "%s: H must be a multiple of 8", fn);
  if (N == 0) return FLCE_OK;
  if (!x || !ckpt) return host_error(FLCE_ERR_ARG, "%s: null pointer", fn);
  if (N > 1 && (x_row < H || x_row >= (int64_t{1} << 38)))
    return host_error(FLCE_ERR_ARG, "%s: row stride must be at least H", fn);
  if (!aligned16(x) || !aligned16(ckpt) || (N > 1 && x_row % 8 != 0))
    return host_error(FLCE_ERR_ALIGN, "%s: buffers must be 16-byte aligned, x_row a multiple of 8",
                      fn);
  if (N * (H / 8) > (int64_t{1} << 40))
    return host_error(FLCE_ERR_ARG, "%s: N * H is too large for one call", fn);
  using wide = __int128;
  const wide e = dtype == FLCE_FP32 ? 4 : 2;
  const wide x0 = reinterpret_cast<uintptr_t>(x), c0 = reinterpret_cast<uintptr_t>(ckpt);
  if (x0 < c0 + flce_ckpt_bytes(N, H) && c0 < x0 + ((N - 1) * wide{x_row} + H) * e)
    return host_error(FLCE_ERR_ARG, "%s: x overlaps the checkpoint", fn);
  return FLCE_OK;
}

int save_or_load(const char* fn, void* x, int64_t x_row, int64_t N, int64_t H, void* ckpt,
                 const flce_opts* opts, bool save) {
  host_clear_error();
  const flce_opts o = opts_or_default(opts);
  int rc = check(fn, x, x_row, N, H, ckpt, o.dtype);
  if (rc) return rc;
  int sms = 0;
  if ((rc = host_device(&sms))) return rc;
  StepCall call;
  if ((rc = call.begin(o, 0, StepCall::kIfAsked))) return rc;
  if (N > 0) {
    const Ckpt c = ckpt_view(ckpt, N, H);
    cudaError_t e;
    if (save) {
      const CkptParams p = params(c, x, x_row, N, H, true);
      if (o.dtype == FLCE_BF16)
        ckpt_save_kernel<bf16_t><<<grid_of(p), kThreads, 0, call.stream>>>(p);
      else
        ckpt_save_kernel<float><<<grid_of(p), kThreads, 0, call.stream>>>(p);
      e = cudaGetLastError();
    } else {
      e = launch_ckpt_load(c, x, x_row, N, H, o.dtype == FLCE_FP32 ? 4 : 2, nullptr,
                           call.stream);
    }
    if (e != cudaSuccess) rc = host_cuda_error(e, fn);
  }
  return call.end(rc);
}

}  // namespace

cudaError_t launch_ckpt_load(const Ckpt& c, void* x, int64_t x_row, int64_t N, int64_t H, int elt,
                             int32_t* clear, cudaStream_t s) {
  CkptParams p = params(c, x, x_row, N, H, false);
  p.clear = clear;
  if (elt == 2)
    ckpt_load_kernel<bf16_t><<<grid_of(p), kThreads, 0, s>>>(p);
  else
    ckpt_load_kernel<float><<<grid_of(p), kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace flce

using namespace flce;

extern "C" {

size_t flce_ckpt_bytes(int64_t N, int64_t H) {
  if (N < 0 || N >= (int64_t{1} << 31) || H < 1 || H > (int64_t{1} << 20)) return 0;
  return static_cast<size_t>(N) * static_cast<size_t>(ckpt_pitch(H) + ckpt_spitch(H));
}

int flce_ckpt_save(const void* x, int64_t x_row, int64_t N, int64_t H, void* ckpt,
                   const flce_opts* opts) {
  return save_or_load("flce_ckpt_save", const_cast<void*>(x), x_row, N, H, ckpt, opts, true);
}

int flce_ckpt_load(const void* ckpt, int64_t N, int64_t H, void* x, int64_t x_row,
                   const flce_opts* opts) {
  return save_or_load("flce_ckpt_load", x, x_row, N, H, const_cast<void*>(ckpt), opts, false);
}

}  // extern "C"
