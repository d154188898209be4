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

// x[j] = x[j] * w + b; either may be missing.
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
__global__ void __launch_bounds__(kFwdThreads, NV == 1 ? 2 : 1)
    resnorm_fwd_kernel(const __grid_constant__ NormParams p) {
  __shared__ float slots[kMaxRowWarps][2][kMaxSums][kMaxRowWarps];
  extern __shared__ __align__(16) uint8_t ring_raw[];
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
  const bool pfp = p.params_fp32, full = p.gate_kind == FLCE_GATE_FULL;
  const bool channel = p.gate_kind == FLCE_GATE_CHANNEL;

  // The ring: of each octet y, then h, then a gate per element.
  const uint32_t step = blockDim.x * 16;
  const uint32_t ring = smem_addr(ring_raw) + threadIdx.x * 16;
  constexpr int kPer = 2 * kPieces<TY> + kPieces<TH>;
  const uint32_t stage = step * NV * kPer;
  auto fetch = [&](int64_t row, int s) {
    if (row < p.N) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (!in[j]) continue;
        const uint32_t at = ring + s * stage + j * kPer * step;
        copy_octet<TY>(at, step, row_at<TY>(p.y.p, row, p.y.row), oct[j]);
        if (p.h.p)
          copy_octet<TH>(at + kPieces<TY> * step, step, row_at<TH>(p.h.p, row, p.h.row), oct[j]);
        if (full)
          copy_octet<TY>(at + (kPieces<TY> + kPieces<TH>) * step, step,
                         row_at<TY>(p.gate.p, row, p.gate.row), oct[j]);
      }
    }
    copies_commit();
  };

  // What multiplies n(y) whatever the row: beta, the weight and a gate per channel; with
  // `b`, what is added (0 without a bias).  And a gate per element.
  auto factor = [&](const void* w, float missing, int o, float (&f)[8]) {
    param_octet<TY>(w, pfp, o, missing, f);
    if (channel) {
      float t[8];
      param_octet<TY>(p.gate.p, pfp, o, 1.f, t);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] *= gate_act(p.act, t[i]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] *= p.beta;
  };
  // A thread with one octet keeps its factors.
  float c[8], w_pre[8];
  if (NV == 1) {
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = w_pre[i] = 0.f;
    if (in[0]) {
      factor(p.w_post, 1.f, oct[0], c);
      param_octet<TY>(p.w_pre, pfp, oct[0], 1.f, w_pre);
    }
  }
  const bool token = p.gate_kind == FLCE_GATE_TOKEN;
  float one = 1.f;  // a gate with one value
  if (p.gate_kind == FLCE_GATE_SCALAR) one = gate_act(p.act, one_element<TY>(p.gate.p, pfp, 0));

  const int64_t first = static_cast<int64_t>(blockIdx.x) * p.groups + group;
  const int64_t rows = static_cast<int64_t>(gridDim.x) * p.groups;
  int s_in = 0, s_out = 0;
  for (; s_in < p.stages - 1; ++s_in) fetch(first + s_in * rows, s_in);
  for (int64_t row = first; row < p.N; row += rows) {
    fetch(row + (p.stages - 1) * rows, s_in);
    s_in = s_in + 1 == p.stages ? 0 : s_in + 1;
    if (token) one = gate_act(p.act, one_element<TY>(p.gate.p, false, row * p.gate.row));
    copies_wait(p.stages - 1);
    const uint32_t at = ring + s_out * stage;
    s_out = s_out + 1 == p.stages ? 0 : s_out + 1;
    float x[NV][8];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[j][i] = 0.f;
      if (in[j]) shared_octet(TY{}, at + j * kPer * step, step, x[j]);
    }
    float mean_y = 0.f, r_y = 0.f, mean_h = 0.f, r_h = 0.f;
    if (p.post) normalise<NV>(x, in, p.layer, p.eps, p.inv_h, sums, mean_y, r_y);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!in[j]) continue;
      const uint32_t mine = at + j * kPer * step;
      float t[8];
      if (NV == 1) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[j][i] *= c[i];
      } else {
        factor(p.w_post, 1.f, oct[j], t);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[j][i] *= t[i];
      }
      if (p.b_post) {
        factor(p.b_post, 0.f, oct[j], t);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[j][i] += t[i];
      }
      if (full) {
        shared_octet(TY{}, mine + (kPieces<TY> + kPieces<TH>) * step, step, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[j][i] *= gate_act(p.act, t[i]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) x[j][i] *= one;
      if (p.h.p) {
        shared_octet(TH{}, mine + kPieces<TY> * step, step, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[j][i] = fmaf(p.alpha, t[i], x[j][i]);
      }
      // the stream is what is stored of it; see flce_resnorm
      const auto o = to_octet(TH{}, x[j]);
      octet_floats(o, x[j]);
      if (p.h_out.p)
        static_cast<typename Elem<TH>::Octet*>(row_at<TH>(p.h_out.p, row, p.h_out.row))[oct[j]] = o;
    }
    if (p.pre) {
      normalise<NV>(x, in, p.layer, p.eps, p.inv_h, sums, mean_h, r_h);
      if (NV == 1) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[0][i] *= w_pre[i];
        affine<TY, NV>(x, in, oct, nullptr, p.b_pre, pfp);
      } else {
        affine<TY, NV>(x, in, oct, p.w_pre, p.b_pre, pfp);
      }
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const auto o = to_octet(TY{}, x[j]);
        if (in[j])
          static_cast<typename Elem<TY>::Octet*>(row_at<TY>(p.z.p, row, p.z.row))[oct[j]] = o;
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
  static SmemLimit limit;
  const int octets = p.H / 8;
  p.warps = (octets + 32 * NV - 1) / (32 * NV);
  p.groups = kFwdThreads / 32 / p.warps;
  const int threads = 32 * p.warps * p.groups;
  const int stage = threads * 16 * NV * (2 * kPieces<TY> + kPieces<TH>);
  // two CTAs on an SM where the registers let them, or one
  int ctas = NV == 1 ? 2 : 1;
  if (ctas == 2 && kSmemPerSm / 2 / stage < 3) ctas = 1;
  p.stages = kSmemPerSm / ctas / stage;
  if (p.stages > 4) p.stages = 4;
  const cudaError_t e = limit.raise(resnorm_fwd_kernel<TY, TH, NV>, kSmemPerSm);
  if (e != cudaSuccess) return e;
  const int64_t want = (p.N + p.groups - 1) / p.groups;
  const int64_t most = static_cast<int64_t>(sms) * ctas;
  resnorm_fwd_kernel<TY, TH, NV><<<static_cast<unsigned>(want < most ? want : most), threads,
                                   static_cast<size_t>(p.stages) * stage, s>>>(p);
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
