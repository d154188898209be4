// resnorm_api.cu -- host side of the residual join: argument checks, launch shape, scratch,
// and the sums over tokens that end the backward pass.
#include <cmath>

#include "host_util.h"
#include "resnorm.h"

namespace flce {
namespace {

constexpr int kSumLanes = 32, kSumRows = 16, kSumAtOnce = 10;

// One thread row takes every kSumRows-th part, kSumAtOnce loads in flight, then the thread
// rows are added in order.
__global__ void __launch_bounds__(kSumLanes * kSumRows)
    resnorm_sums_kernel(const __grid_constant__ NormSums p) {
  __shared__ float s[kSumRows][kSumLanes + 1];
  const int k = blockIdx.y, lane = threadIdx.x % kSumLanes, ty = threadIdx.x / kSumLanes;
  const int col = blockIdx.x * kSumLanes + lane;
  grid_dependency_wait();
  if (blockIdx.x * kSumLanes >= static_cast<unsigned>(p.width[k])) return;
  float v = 0.f;
  if (col < p.width[k]) {
    const float* at = p.part[k] + col;
    for (int64_t i = ty; i < p.parts; i += kSumRows * kSumAtOnce) {
      float t[kSumAtOnce];
#pragma unroll
      for (int j = 0; j < kSumAtOnce; ++j) {
        const int64_t n = i + j * kSumRows;
        t[j] = n < p.parts ? at[n * p.width[k]] : 0.f;
      }
#pragma unroll
      for (int j = 0; j < kSumAtOnce; ++j) v += t[j];
    }
  }
  s[ty][lane] = v;
  __syncthreads();
  if (ty != 0 || col >= p.width[k]) return;
  for (int i = 1; i < kSumRows; ++i) v += s[i][lane];
  p.out[k][col] = v;
}

}  // namespace

cudaError_t launch_resnorm_sums(const NormSums& p, cudaStream_t s) {
  int most = 0;
  for (int k = 0; k < 5; ++k) most = p.width[k] > most ? p.width[k] : most;
  if (most == 0) return cudaSuccess;
  // its CTAs may start while the rows' kernel ends
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(static_cast<unsigned>((most + kSumLanes - 1) / kSumLanes), 5);
  cfg.blockDim = dim3(kSumLanes * kSumRows);
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.parts > 0 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, resnorm_sums_kernel, p);
}

namespace {

using wide = __int128;

// Bytes of a tensor: `rows` rows of `width` bytes, `pitch` apart.
struct Span {
  const char* name;
  const void* p;
  wide pitch, width, rows;
};

// Whether two tensors share a byte, where that can be told; rows that interleave at equal
// pitches share none.
bool shared(const Span& a, const Span& b) {
  if (!a.p || !b.p || a.rows == 0 || b.rows == 0) return false;
  const wide a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  if (a0 + (a.rows - 1) * a.pitch + a.width <= b0 || b0 + (b.rows - 1) * b.pitch + b.width <= a0)
    return false;
  if (a.rows > 1 && b.rows > 1 && a.pitch == b.pitch) {
    const wide off = ((b0 - a0) % a.pitch + a.pitch) % a.pitch;
    return !(off >= a.width && off + b.width <= a.pitch);
  }
  return true;
}

int check_row(const char* name, const void* p, int64_t& stride, int64_t N, int64_t H) {
  if (!p) return host_error(FLCE_ERR_ARG, "%s is null", name);
  if (N <= 1) stride = H;
  if (stride < H || stride >= (int64_t{1} << 38))
    return host_error(FLCE_ERR_ARG, "%s: row stride must be at least H", name);
  if (stride % 8 != 0 || !aligned16(p))
    return host_error(FLCE_ERR_ALIGN,
                      "%s must be 16-byte aligned with a row stride that is a multiple of 8", name);
  return FLCE_OK;
}

int check_vec(const char* name, const void* p) {
  if (!aligned16(p)) return host_error(FLCE_ERR_ALIGN, "%s must be 16-byte aligned", name);
  return FLCE_OK;
}

int resnorm(const flce_resnorm* in, const flce_opts* opts, bool backward) {
  host_clear_error();
  const flce_opts o = opts_or_default(opts);
  if (!in) return host_error(FLCE_ERR_ARG, "null flce_resnorm");
  flce_resnorm a = *in;
  if (backward) {
    a.h = nullptr;
    a.z = a.z_ckpt = nullptr;
  } else {
    a.dz = a.dh_out = nullptr;
    a.dy = a.dh = nullptr;
  }
  // a norm that there is not has no parameters: the forward kernel takes what is given
  if (!a.post_norm) a.w_post = a.b_post = nullptr;
  if (!a.pre_norm) a.w_pre = a.b_pre = nullptr;
  if (o.dtype != FLCE_BF16 && o.dtype != FLCE_FP32)
    return host_error(FLCE_ERR_ARG, "unknown dtype %d", o.dtype);
  if (a.N < 0 || a.N >= (int64_t{1} << 31))
    return host_error(FLCE_ERR_ARG, "N must be in 0 .. 2^31 - 1");
  if (a.H < 8 || a.H > kMaxH || a.H % 8 != 0)
    return host_error(FLCE_ERR_ARG, "H must be a multiple of 8 in 8 .. %d (got %lld)", kMaxH,
                      static_cast<long long>(a.H));
  if (a.norm != FLCE_NORM_RMS && a.norm != FLCE_NORM_LAYER)
    return host_error(FLCE_ERR_ARG, "unknown norm %d", a.norm);
  if (a.gate_kind < FLCE_GATE_NONE || a.gate_kind > FLCE_GATE_FULL)
    return host_error(FLCE_ERR_ARG, "unknown gate kind %d", a.gate_kind);
  if (a.gate_act < FLCE_ACT_NONE || a.gate_act > FLCE_ACT_TANH)
    return host_error(FLCE_ERR_ARG, "unknown gate activation %d", a.gate_act);
  if (!std::isfinite(a.alpha) || !std::isfinite(a.beta))
    return host_error(FLCE_ERR_ARG, "alpha and beta must be finite");
  if (!(a.eps >= 0.f) || std::isinf(a.eps))
    return host_error(FLCE_ERR_ARG, "eps must be finite and not negative");
  const int64_t N = a.N, H = a.H;
  const wide ey = o.dtype == FLCE_FP32 ? 4 : 2;
  const wide eh = ey == 4 || a.stream_fp32 ? 4 : 2, ep = ey == 4 || a.params_fp32 ? 4 : 2;
  const bool gated = a.gate_kind != FLCE_GATE_NONE;
  const bool token = a.gate_kind == FLCE_GATE_TOKEN, full = a.gate_kind == FLCE_GATE_FULL;
  int rc = FLCE_OK;
  auto elem = [&](const char* name, const void* p, wide bytes) {
    if (!p) return host_error(FLCE_ERR_ARG, "%s is null", name);
    if (reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(bytes))
      return host_error(FLCE_ERR_ALIGN, "%s must be aligned to its element", name);
    return static_cast<int>(FLCE_OK);
  };
  // gates: without tokens only those that are parameters have memory
  auto gate = [&](const char* name, const void* p, int64_t& stride, wide param_bytes) {
    if (a.gate_kind == FLCE_GATE_SCALAR) return elem(name, p, param_bytes);
    if (a.gate_kind == FLCE_GATE_CHANNEL)
      return p ? check_vec(name, p) : host_error(FLCE_ERR_ARG, "%s is null", name);
    if (N == 0) return static_cast<int>(FLCE_OK);
    if (full) return check_row(name, p, stride, N, H);
    if (N == 1) stride = 1;
    if (stride < 1 || stride >= (int64_t{1} << 38))
      return host_error(FLCE_ERR_ARG, "%s: row stride must be positive", name);
    return elem(name, p, ey);
  };
  struct { const char* name; const void* p; } vecs[] = {
      {"w_post", a.w_post}, {"b_post", a.b_post}, {"w_pre", a.w_pre}, {"b_pre", a.b_pre}};
  for (const auto& v : vecs)
    if ((rc = check_vec(v.name, v.p))) return rc;
  if (gated && (rc = gate("gate", a.gate, a.gate_row, ep))) return rc;
  const bool reads_y = !backward || a.post_norm || gated;
  if (N > 0) {
    if (reads_y && (rc = check_row("y", a.y, a.y_row, N, H))) return rc;
    if (!backward) {
      if (a.h && (rc = check_row("h", a.h, a.h_row, N, H))) return rc;
      if (a.h_out && (rc = check_row("h_out", a.h_out, a.h_out_row, N, H))) return rc;
      if (a.pre_norm && (rc = check_row("z", a.z, a.z_row, N, H))) return rc;
      if (!a.pre_norm && !a.h_out) return host_error(FLCE_ERR_ARG, "h_out is null");
      if (a.stats && (rc = elem("stats", a.stats, 4))) return rc;
      if (a.z_ckpt && !a.pre_norm)
        return host_error(FLCE_ERR_ARG, "a checkpoint of z needs pre_norm");
      if ((rc = check_vec("z_ckpt", a.z_ckpt))) return rc;
    } else {
      if (a.pre_norm) {
        if ((rc = check_row("dz", a.dz, a.dz_row, N, H))) return rc;
        if ((rc = check_row("h_out", a.h_out, a.h_out_row, N, H))) return rc;
      }
      if (a.pre_norm || a.post_norm)
        if ((rc = elem("stats", a.stats, 4))) return rc;
      if (a.dh_out && (rc = check_row("dh_out", a.dh_out, a.dh_out_row, N, H))) return rc;
      if (!a.pre_norm && !a.dh_out)
        return host_error(FLCE_ERR_ARG, "neither dz nor dh_out is given");
      if ((rc = check_row("dy", a.dy, a.dy_row, N, H))) return rc;
      if (a.dh && (rc = check_row("dh", a.dh, a.dh_row, N, H))) return rc;
    }
  }
  struct { const char* name; float* p; int32_t width; } sums[] = {
      {"dw_pre", a.pre_norm ? a.dw_pre : nullptr, static_cast<int32_t>(H)},
      {"db_pre", a.pre_norm ? a.db_pre : nullptr, static_cast<int32_t>(H)},
      {"dw_post", a.post_norm ? a.dw_post : nullptr, static_cast<int32_t>(H)},
      {"db_post", a.post_norm ? a.db_post : nullptr, static_cast<int32_t>(H)},
      {"dgate", gated && !token && !full ? static_cast<float*>(a.dgate) : nullptr,
       a.gate_kind == FLCE_GATE_SCALAR ? 1 : static_cast<int32_t>(H)}};
  if (backward) {
    if (gated && (rc = gate("dgate", a.dgate, a.dgate_row, 4))) return rc;
    for (int k = 0; k < 4; ++k)
      if ((rc = check_vec(sums[k].name, sums[k].p))) return rc;
  }
  // overlaps: what a thread writes, only itself may have read, and before
  auto rows = [&](const char* name, const void* p, int64_t stride, wide e) {
    return Span{name, p, stride * e, H * e, N};
  };
  auto vec = [&](const char* name, const void* p, wide bytes) {
    return Span{name, p, bytes, bytes, 1};
  };
  const Span gate_in = !gated ? Span{} : full ? rows("gate", a.gate, a.gate_row, ey)
                       : token ? Span{"gate", a.gate, a.gate_row * ey, ey, N}
                       : vec("gate", a.gate, a.gate_kind == FLCE_GATE_SCALAR ? ep : H * ep);
  Span ins[10], outs[8];
  int ni = 0, no = 0;
  if (reads_y) ins[ni++] = rows("y", a.y, a.y_row, ey);
  if (gated) ins[ni++] = gate_in;
  for (const auto& v : vecs) ins[ni++] = vec(v.name, v.p, H * ep);
  if (!backward) {
    ins[ni++] = rows("h", a.h, a.h_row, eh);
    outs[no++] = rows("h_out", a.h_out, a.h_out_row, eh);
    if (a.pre_norm) outs[no++] = rows("z", a.z, a.z_row, ey);
    outs[no++] = vec("stats", a.stats, N * 16);
    if (a.z_ckpt) outs[no++] = vec("z_ckpt", a.z_ckpt, flce_ckpt_bytes(N, H));
  } else {
    if (a.pre_norm) {
      ins[ni++] = rows("dz", a.dz, a.dz_row, ey);
      ins[ni++] = rows("h_out", a.h_out, a.h_out_row, eh);
    }
    if (a.pre_norm || a.post_norm) ins[ni++] = vec("stats", a.stats, N * 16);
    ins[ni++] = rows("dh_out", a.dh_out, a.dh_out_row, eh);
    outs[no++] = rows("dy", a.dy, a.dy_row, ey);
    outs[no++] = rows("dh", a.dh, a.dh_row, eh);
    if (full) outs[no++] = rows("dgate", a.dgate, a.dgate_row, ey);
    if (token) outs[no++] = Span{"dgate", a.dgate, a.dgate_row * ey, ey, N};
    for (const auto& v : sums)
      if (v.p) outs[no++] = vec(v.name, v.p, v.width * wide{4});
  }
  for (int i = 0; N > 0 && i < no; ++i) {
    for (int j = 0; j < ni; ++j) {
      // (fields of the other pass are null here, and so is no tensor that is compared)
      const bool in_place = outs[i].p == ins[j].p && outs[i].pitch == ins[j].pitch &&
                            outs[i].width == ins[j].width;
      const bool may = (outs[i].p == a.h_out && ins[j].p == a.h) ||
                       (outs[i].p == a.z && ins[j].p == a.y) ||
                       (outs[i].p == a.dh && ins[j].p == a.dh_out) ||
                       (outs[i].p == a.dy && ins[j].p == a.dz);
      if (in_place && may) continue;
      if (shared(outs[i], ins[j]))
        return host_error(FLCE_ERR_ARG, "%s overlaps %s", outs[i].name, ins[j].name);
    }
    for (int j = 0; j < i; ++j)
      if (shared(outs[i], outs[j]))
        return host_error(FLCE_ERR_ARG, "%s overlaps %s", outs[i].name, outs[j].name);
  }

  int sms = 0;
  if ((rc = host_device(&sms))) return rc;
  NormParams p{};
  p.N = N;
  p.H = static_cast<int32_t>(H);
  p.layer = a.norm == FLCE_NORM_LAYER;
  p.post = a.post_norm != 0;
  p.pre = a.pre_norm != 0;
  p.params_fp32 = ep == 4;
  p.gate_kind = a.gate_kind;
  p.act = a.gate_act;
  p.alpha = a.alpha;
  p.beta = a.beta;
  p.eps = a.eps;
  p.inv_h = 1.f / static_cast<float>(H);
  auto row = [](const void* q, int64_t stride) { return RowTensor{const_cast<void*>(q), stride, 0}; };
  p.y = row(a.y, a.y_row);
  p.gate = row(a.gate, a.gate_row);
  p.w_post = a.w_post;
  p.b_post = a.b_post;
  p.w_pre = a.w_pre;
  p.b_pre = a.b_pre;
  p.h_out = row(a.h_out, a.h_out_row);
  p.stats = a.stats;
  p.wide = 1;
  for (const void* q : {static_cast<const void*>(backward ? a.dy : a.h_out),
                        static_cast<const void*>(backward ? a.dh : a.z),
                        static_cast<const void*>(full ? a.dgate : nullptr)})
    if (reinterpret_cast<uintptr_t>(q) & 31) p.wide = 0;
  StepCall call;
  if (!backward) {
    p.h = row(a.h, a.h_row);
    p.z = row(a.z, a.z_row);
    if (a.z_ckpt) p.ckpt = ckpt_view(a.z_ckpt, N, H);
    if ((rc = call.begin(o, 0, StepCall::kIfAsked))) return rc;
    if (N > 0) {
      const cudaError_t e =
          ey == 4   ? launch_resnorm_fwd_fp32(p, sms, call.stream)
          : eh == 4 ? launch_resnorm_fwd_mixed(p, sms, call.stream)
                    : launch_resnorm_fwd_bf16(p, sms, call.stream);
      if (e != cudaSuccess) rc = host_cuda_error(e, "resnorm_fwd");
    }
    return call.end(rc);
  }
  p.dz = row(a.dz, a.dz_row);
  p.dh_out = row(a.dh_out, a.dh_out_row);
  p.dy = row(a.dy, a.dy_row);
  p.dh = row(a.dh, a.dh_row);
  p.dgate = row(a.dgate, a.dgate_row);
  // what of it a row's kernel is to make decides between its variants, hence its shape
  auto rows_kernel = [&](int64_t parts) {
    return ey == 4   ? launch_resnorm_bwd_fp32(p, parts, call.stream)
           : eh == 4 ? launch_resnorm_bwd_mixed(p, parts, call.stream)
                     : launch_resnorm_bwd_bf16(p, parts, call.stream);
  };
  p.biased = a.norm == FLCE_NORM_LAYER || (a.post_norm && (a.b_post || a.db_post)) ||
             (a.pre_norm && a.db_pre);
  int64_t parts = 0;
  if (N > 0) {
    p.sms = sms;
    const cudaError_t e = rows_kernel(0);
    if (e != cudaSuccess) return host_cuda_error(e, "resnorm_bwd");
    const int64_t want = (N + p.groups - 1) / p.groups;
    parts = want < p.fit ? want : p.fit;
  }
  size_t at[5], bytes = 0;
  for (int k = 0; k < 5; ++k) {
    at[k] = bytes;
    if (sums[k].p) bytes += round256(static_cast<size_t>(parts) * static_cast<size_t>(sums[k].width) * 4);
  }
  if ((rc = call.begin(o, bytes, StepCall::kIfAsked))) return rc;
  NormSums t{};
  t.parts = parts;
  for (int k = 0; k < 5; ++k) {
    if (!sums[k].p) continue;
    p.part[k] = reinterpret_cast<float*>(call.scratch + at[k]);
    t.part[k] = p.part[k];
    t.out[k] = sums[k].p;
    t.width[k] = sums[k].width;
    p.sums_follow = 1;
  }
  cudaError_t e = cudaSuccess;
  if (N > 0) e = rows_kernel(parts);
  if (e == cudaSuccess) e = launch_resnorm_sums(t, call.stream);
  if (e != cudaSuccess) rc = host_cuda_error(e, "resnorm_bwd");
  return call.end(rc);
}

}  // namespace
}  // namespace flce

using namespace flce;

extern "C" {

int flce_resnorm_fwd(const flce_resnorm* a, const flce_opts* opts) {
  return resnorm(a, opts, false);
}

int flce_resnorm_bwd(const flce_resnorm* a, const flce_opts* opts) {
  return resnorm(a, opts, true);
}

size_t flce_resnorm_sizeof(void) { return sizeof(flce_resnorm); }

}  // extern "C"
