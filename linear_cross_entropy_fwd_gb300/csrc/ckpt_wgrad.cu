// ckpt_wgrad.cu -- a projection's weight gradient from its input's 8-bit checkpoint:
// dW [O, I] (+)= dY^T X, dY [N, O] bf16, X [N, I] as ckpt.cuh stores it.
#include "ckpt.cuh"
#include "host_util.h"
#include "launch.h"

namespace flce {
namespace {

int check(const void* dY, int64_t dY_row, const void* ckpt, int64_t N, int64_t O, int64_t I,
          const float* dW, int32_t dtype) {
  const char* fn = "flce_ckpt_wgrad";
  if (dtype != FLCE_BF16) return host_error(FLCE_ERR_ARG, "%s takes bf16 dY (dtype %d)", fn, dtype);
  const int64_t most = int64_t{1} << 20;
  if (N < 0 || N >= (int64_t{1} << 31) || O < 1 || O > most || I < 1 || I > most)
    return host_error(FLCE_ERR_ARG, "%s: sizes must satisfy 0 <= N < 2^31, 1 <= O, I <= 2^20", fn);
  if (O % 8 != 0 || I % 8 != 0)
    return host_error(FLCE_ERR_ALIGN, "%s: O and I must be multiples of 8", fn);
  if (!dW || (N > 0 && (!dY || !ckpt))) return host_error(FLCE_ERR_ARG, "%s: null pointer", fn);
  if (!aligned16(dW)) return host_error(FLCE_ERR_ALIGN, "%s: dW must be 16-byte aligned", fn);
  if (N == 0) return FLCE_OK;
  if (N > 1 && (dY_row < O || dY_row >= (int64_t{1} << 38)))
    return host_error(FLCE_ERR_ARG, "%s: row stride must be at least O", fn);
  if (!aligned16(dY) || !aligned16(ckpt) || (N > 1 && dY_row % 8 != 0))
    return host_error(FLCE_ERR_ALIGN,
                      "%s: buffers must be 16-byte aligned, dY_row a multiple of 8", fn);
  using wide = __int128;
  const wide w0 = reinterpret_cast<uintptr_t>(dW), w1 = w0 + wide{O} * I * 4;
  const wide y0 = reinterpret_cast<uintptr_t>(dY), c0 = reinterpret_cast<uintptr_t>(ckpt);
  if ((w0 < y0 + ((N - 1) * wide{dY_row} + O) * 2 && y0 < w1) ||
      (w0 < c0 + flce_ckpt_bytes(N, I) && c0 < w1))
    return host_error(FLCE_ERR_ARG, "%s: dW overlaps an input", fn);
  return FLCE_OK;
}

int map_of(CUtensorMap* m, const void* p, CUtensorMapDataType t, int64_t cols, int64_t rows,
           int64_t pitch, uint32_t box_cols, uint32_t box_rows, const char* what) {
  const uint64_t dims[2] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(rows)};
  const uint64_t pitches[1] = {static_cast<uint64_t>(pitch)};
  const uint32_t box[2] = {box_cols, box_rows};
  return host_tensor_map(m, p, t, 2, dims, pitches, box, what);
}

}  // namespace
}  // namespace flce

using namespace flce;

extern "C" int flce_ckpt_wgrad(const void* dY, int64_t dY_row, const void* ckpt, int64_t N,
                               int64_t O, int64_t I, float* dW, int32_t accumulate,
                               const flce_opts* opts) {
  host_clear_error();
  const flce_opts o = opts_or_default(opts);
  int rc = check(dY, dY_row, ckpt, N, O, I, dW, o.dtype);
  if (rc) return rc;
  int sms = 0;
  if ((rc = host_device(&sms))) return rc;
  StepCall call;
  if ((rc = call.begin(o, N > 0 ? round256(static_cast<size_t>(N) * I * 2) : 0, StepCall::kCleared)))
    return rc;
  if (N == 0) {
    if (!accumulate) {
      const cudaError_t e =
          cudaMemsetAsync(dW, 0, static_cast<size_t>(O) * static_cast<size_t>(I) * 4, call.stream);
      if (e != cudaSuccess) rc = host_cuda_error(e, "cudaMemsetAsync(dW)");
    }
    return call.end(rc);
  }
  CUtensorMap ma, mb, mw;
  int units = 0;
  cudaError_t e = gemm_prepare_bf16(sms, &units);
  if (e != cudaSuccess) return call.end(host_cuda_error(e, "gemm_prepare"));
  if ((rc = map_of(&ma, dY, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, O, N, (N > 1 ? dY_row : O) * 2, 64,
                   64, "dY")) ||
      (rc = map_of(&mb, call.scratch, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, I, N, I * 2, 64, 64,
                   "X")) ||
      (rc = map_of(&mw, dW, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, I, O, I * 4, 32, 32, "dW")))
    return call.end(rc);
  e = launch_ckpt_load(ckpt_view(const_cast<void*>(ckpt), N, I), call.scratch, I, N, I, 2,
                       call.stream);
  if (e == cudaSuccess) {
    GemmGrid g{};
    g.num_m_blk = static_cast<int32_t>((O + 2 * BM - 1) / (2 * BM));
    g.num_n_blk = static_cast<int32_t>((I + BN - 1) / BN);
    g.num_k_blk = static_cast<int32_t>((N + 63) / 64);
    g.raster_n = 1;
    g.wait_operands = 1;
    g.status = call.status;
    const int64_t tiles = static_cast<int64_t>(g.num_m_blk) * g.num_n_blk;
    const StoreParams sp{0, 0, accumulate ? 1 : 0};
    e = launch_dw_bf16(ma, mb, mw, g, sp, static_cast<int>(tiles < units ? tiles : units),
                       call.stream);
  }
  if (e != cudaSuccess) rc = host_cuda_error(e, "ckpt_wgrad");
  return call.end(rc);
}
