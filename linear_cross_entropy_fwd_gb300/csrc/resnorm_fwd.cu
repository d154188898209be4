// resnorm_fwd.cu -- the residual join's forward pass (resnorm.h has the formulas).
//
// Bound by memory: a token's y and h are read once and h', z written once.  `warps` warps
// hold a row in registers, NV octets a thread, and a CTA has several rows at a time when
// they are short.  A mean and a variance are two sums one after the other, so that nothing
// cancels; RMS norms need one.  A row may hold anything finite.
#include "host_util.h"
#include "resnorm.h"

namespace flce {
namespace {

constexpr int kFwdThreads = 512;

// Sum of (x - mean)^2 over the row; places behind its end hold 0 and stay out of it.
template <int NV>
__device__ __forceinline__ float squares(const float (&x)[NV][8], const bool (&in)[NV], float mean,
                                         RowSums& sums) {
  float s[1] = {0.f};
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float d = in[j] ? x[j][i] - mean : 0.f;
      s[0] = fmaf(d, d, s[0]);
    }
  sums.add(s);
  return s[0];
}

template <int NV>
__device__ __forceinline__ float mean_of(const float (&x)[NV][8], float inv_h, RowSums& sums) {
  float s[1] = {0.f};
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) s[0] += x[j][i];
  sums.add(s);
  return s[0] * inv_h;
}

// x -> n(x) in place over the row; mean and r for the statistics.
template <int NV>
__device__ __forceinline__ void normalise(float (&x)[NV][8], const bool (&in)[NV], bool layer,
                                          float eps, float inv_h, RowSums& sums, float& mean,
                                          float& r) {
  mean = layer ? mean_of<NV>(x, inv_h, sums) : 0.f;
  float v = fmaf(squares<NV>(x, in, mean, sums), inv_h, eps);
  float m = mean, scale = 1.f;
  if (!(v < 1e38f) || v < 1e-30f) {
    // Squares beyond fp32's range: the row times a power of two, whose squares are not.  (With
    // an eps above 1e-30, squares that vanish beside it need nothing.)
    float top = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[j][i]));
    top = sums.max(top);
    const int k = min(max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -100), 126);
    scale = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) x[j][i] *= scale;
    m = layer ? mean_of<NV>(x, inv_h, sums) : 0.f;
    v = fmaf(squares<NV>(x, in, m, sums), inv_h, eps * scale * scale);
    mean = m / scale;
  }
  r = rsqrtf(v);
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) x[j][i] = in[j] ? (x[j][i] - m) * r : 0.f;
  r *= scale;
}

template <class T, int NV>
__device__ __forceinline__ void affine(float (&x)[NV][8], const bool (&in)[NV],
                                       const int (&oct)[NV], const void* w, const void* b,
                                       bool fp32) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (!in[j]) continue;
    float t[8];
    if (w) {
      param_octet<T>(w, fp32, oct[j], 1.f, t);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[j][i] *= t[i];
    }
    if (b) {
      param_octet<T>(b, fp32, oct[j], 0.f, t);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[j][i] += t[i];
    }
  }
}

template <class TY, class TH, int NV>
__global__ void __launch_bounds__(kFwdThreads, NV == 4 ? 1 : 2)
    resnorm_fwd_kernel(const __grid_constant__ NormParams p) {
  __shared__ float slots[kMaxRowWarps][2][kMaxSums][kMaxRowWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int group = warp / p.warps;
  RowSums sums{slots[group], p.warps, warp - group * p.warps, group, 0};
  for (int i = threadIdx.x; i < kMaxRowWarps * 2 * kMaxSums * kMaxRowWarps; i += blockDim.x)
    (&slots[0][0][0][0])[i] = 0.f;
  __syncthreads();
  const int octets = p.H / 8;
  int oct[NV];
  bool in[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    oct[j] = (j * p.warps + sums.warp) * 32 + lane;
    in[j] = oct[j] < octets;
  }
  const bool pfp = p.params_fp32;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * p.groups + group; row < p.N;
       row += static_cast<int64_t>(gridDim.x) * p.groups) {
    float x[NV][8], hv[NV][8];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[j][i] = hv[j][i] = 0.f;
      if (in[j]) {
        octet_floats(load_octet<TY>(row_at<TY>(p.y.p, row, p.y.row), oct[j]), x[j]);
        if (p.h.p) octet_floats(load_octet<TH>(row_at<TH>(p.h.p, row, p.h.row), oct[j]), hv[j]);
      }
    }
    float mean_y = 0.f, r_y = 0.f, mean_h = 0.f, r_h = 0.f;
    if (p.post) {
      normalise<NV>(x, in, p.layer, p.eps, p.inv_h, sums, mean_y, r_y);
      affine<TY, NV>(x, in, oct, p.w_post, p.b_post, pfp);
    }
    if (p.gate_kind != FLCE_GATE_NONE) {
      float a = 0.f;
      if (p.gate_kind == FLCE_GATE_SCALAR)
        a = gate_act(p.act, one_element<TY>(p.gate.p, pfp, 0));
      else if (p.gate_kind == FLCE_GATE_TOKEN)
        a = gate_act(p.act, one_element<TY>(p.gate.p, false, row * p.gate.row));
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (!in[j]) continue;
        float t[8];
        if (p.gate_kind == FLCE_GATE_CHANNEL)
          param_octet<TY>(p.gate.p, pfp, oct[j], 1.f, t);
        else if (p.gate_kind == FLCE_GATE_FULL)
          octet_floats(load_octet<TY>(row_at<TY>(p.gate.p, row, p.gate.row), oct[j]), t);
        const bool each = p.gate_kind == FLCE_GATE_CHANNEL || p.gate_kind == FLCE_GATE_FULL;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[j][i] *= each ? gate_act(p.act, t[i]) : a;
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[j][i] = fmaf(p.alpha, hv[j][i], p.beta * x[j][i]);
      // the stream is what is stored of it; see flce_resnorm
      const auto o = to_octet(TH{}, x[j]);
      octet_floats(o, x[j]);
      if (in[j] && p.h_out.p)
        static_cast<typename Elem<TH>::Octet*>(row_at<TH>(p.h_out.p, row, p.h_out.row))[oct[j]] = o;
    }
    if (p.pre) {
      normalise<NV>(x, in, p.layer, p.eps, p.inv_h, sums, mean_h, r_h);
      affine<TY, NV>(x, in, oct, p.w_pre, p.b_pre, pfp);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const auto o = to_octet(TY{}, x[j]);
        if (in[j]) static_cast<typename Elem<TY>::Octet*>(row_at<TY>(p.z.p, row, p.z.row))[oct[j]] = o;
        if (p.ckpt.codes) {
          octet_floats(o, x[j]);
          ckpt_store_octet(p.ckpt, row, oct[j], x[j]);
        }
      }
    }
    if (p.stats && lane == 0 && sums.warp == 0) {
      p.stats[row] = mean_y;
      p.stats[p.N + row] = r_y;
      p.stats[2 * p.N + row] = mean_h;
      p.stats[3 * p.N + row] = r_h;
    }
  }
}

template <class TY, class TH, int NV>
cudaError_t launch(NormParams p, int sms, cudaStream_t s) {
  const int octets = p.H / 8;
  p.warps = (octets + 32 * NV - 1) / (32 * NV);
  p.groups = kFwdThreads / 32 / p.warps;
  const int64_t want = (p.N + p.groups - 1) / p.groups;
  const int64_t most = static_cast<int64_t>(sms) * (NV == 4 ? 1 : 2);
  resnorm_fwd_kernel<TY, TH, NV>
      <<<static_cast<unsigned>(want < most ? want : most), 32 * p.warps * p.groups, 0, s>>>(p);
  return cudaGetLastError();
}

template <class TY, class TH>
cudaError_t launch_nv(const NormParams& p, int sms, cudaStream_t s) {
  if (p.H <= 4096) return launch<TY, TH, 1>(p, sms, s);
  return p.H <= 8192 ? launch<TY, TH, 2>(p, sms, s) : launch<TY, TH, 4>(p, sms, s);
}

}  // namespace

cudaError_t launch_resnorm_fwd(const NormParams& p, int y_bytes, int h_bytes, int sms,
                               cudaStream_t s) {
  if (y_bytes == 4) return launch_nv<float, float>(p, sms, s);
  return h_bytes == 4 ? launch_nv<bf16_t, float>(p, sms, s) : launch_nv<bf16_t, bf16_t>(p, sms, s);
}

}  // namespace flce
