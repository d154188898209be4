// resnorm_bwd.cuh -- the residual join's backward pass (resnorm.h has the formulas); one
// translation unit per pair of types includes it.
//
// A thread has the same 8 columns of every row that its warps take, so that the sums over
// tokens stay in its registers until the end, one fp32 row for each group of warps; a second
// kernel adds those in a fixed order.  Rows of more than 4096 elements are shared by the
// CTAs of a cluster for the same reason: 8 columns a thread is what 5 such sums leave room for.
//
// The two norms' sums would follow one another (the post-norm's need dt, dt needs the
// pre-norm's).  But dt is linear in them: with e = dh' + r g and q = beta a w_post,
//   dt = e - r m1 - r m2 xh,   sum gy yh = sum q yh e - r m1 sum q yh - r m2 sum q yh xh
// (and the same without yh), so all sums of a row are taken together, one exchange per row.
#pragma once
#include "host_util.h"
#include "resnorm.h"

namespace flce {

constexpr int kBwdThreads = 512;

// Gates as the kernel tells them apart.
enum { kNoGate = 0, kOneGate = 1 /* of a token or of all */, kChannelGate = 2, kFullGate = 3 };

// Sums over the CTAs of a cluster that share a row: every CTA puts its own in every CTA's
// slots.  Two sets in turn, as in RowSums.
struct ClusterSums {
  float (*slots)[4][kMaxSums];  // [2]
  int ctas, rank;
  uint32_t turn;

  template <int K>
  __device__ __forceinline__ void add(float (&v)[K]) {
    if (ctas == 1) return;
    float(*s)[kMaxSums] = slots[turn & 1];
    ++turn;
    if (threadIdx.x < static_cast<uint32_t>(ctas)) {
      const uint32_t to = mapa_shared(smem_addr(&s[rank][0]), threadIdx.x);
#pragma unroll
      for (int k = 0; k < K; ++k)
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + 4 * k), "f"(v[k]) : "memory");
    }
    cluster_sync();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      v[k] = s[0][k];
      for (int c = 1; c < ctas; ++c) v[k] += s[c][k];
    }
  }
};

// AFF: a mean or a bias is wanted.
template <class TY, class TH, bool POST, bool AFF, int GATE>
__global__ void __launch_bounds__(kBwdThreads, 1)
    resnorm_bwd_kernel(const __grid_constant__ NormParams p) {
  __shared__ float slots[kMaxRowWarps][2][kMaxSums][kMaxRowWarps];
  __shared__ float cluster_slots[2][4][kMaxSums];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int group = warp / p.warps;
  const int rank = p.cluster > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  RowSums sums{slots[group], p.warps, warp - group * p.warps, group, 0};
  ClusterSums more{cluster_slots, p.cluster, rank, 0};
  for (int i = threadIdx.x; i < kMaxRowWarps * 2 * kMaxSums * kMaxRowWarps; i += blockDim.x)
    (&slots[0][0][0][0])[i] = 0.f;
  __syncthreads();
  if (p.cluster > 1) cluster_sync();  // every CTA runs before its slots are written
  const int in_cta = sums.warp * 32 + lane;
  const int oct = rank * p.octets + in_cta;
  const bool in = in_cta < p.octets && oct < p.H / 8;
  const bool pfp = p.params_fp32, layer = p.layer;

  float w_pre[8], w_post[8], b_post[8], a[8], slope[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w_pre[i] = w_post[i] = b_post[i] = a[i] = slope[i] = 0.f;
  if (in) {
    param_octet<TY>(p.w_pre, pfp, oct, 1.f, w_pre);
    if (POST) param_octet<TY>(p.w_post, pfp, oct, 1.f, w_post);
    if (POST && AFF) param_octet<TY>(p.b_post, pfp, oct, 0.f, b_post);
    if (GATE == kChannelGate) param_octet<TY>(p.gate.p, pfp, oct, 1.f, a);
  }
  if (GATE == kOneGate && p.gate_kind == FLCE_GATE_SCALAR) a[0] = one_element<TY>(p.gate.p, pfp, 0);
  if (GATE == kChannelGate || GATE == kOneGate) {
#pragma unroll
    for (int i = 0; i < (GATE == kOneGate ? 1 : 8); ++i) {
      a[i] = gate_act(p.act, a[i]);
      slope[i] = p.beta * gate_slope(p.act, a[i]);
      a[i] *= p.beta;
    }
  }

  float s_wpre[8], s_bpre[8], s_wpost[8], s_bpost[8], s_gate[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) s_wpre[i] = s_bpre[i] = s_wpost[i] = s_bpost[i] = s_gate[i] = 0.f;

  const int64_t unit = static_cast<int64_t>(blockIdx.x / p.cluster) * p.groups + group;
  const int64_t units = static_cast<int64_t>(gridDim.x / p.cluster) * p.groups;
  for (int64_t row = unit; row < p.N; row += units) {
    float dz[8], xh[8], e[8], yh[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) dz[i] = xh[i] = e[i] = yh[i] = 0.f;
    float mean_y = 0.f, r_y = 1.f, r_h = 0.f;
    if (POST) {
      mean_y = p.stats[row];
      r_y = p.stats[p.N + row];
    }
    if (p.pre) {
      const float mean_h = p.stats[2 * p.N + row];
      r_h = p.stats[3 * p.N + row];
      if (in) {
        octet_floats(load_octet<TY>(row_at<TY>(p.dz.p, row, p.dz.row), oct), dz);
        octet_floats(load_octet<TH>(row_at<TH>(p.h_out.p, row, p.h_out.row), oct), xh);
#pragma unroll
        for (int i = 0; i < 8; ++i) xh[i] = (xh[i] - mean_h) * r_h;
      }
    }
    if (in) {
      if (p.dh_out.p) octet_floats(load_octet<TH>(row_at<TH>(p.dh_out.p, row, p.dh_out.row), oct), e);
      if (POST || GATE != kNoGate) {
        octet_floats(load_octet<TY>(row_at<TY>(p.y.p, row, p.y.row), oct), yh);
        if (POST) {
#pragma unroll
          for (int i = 0; i < 8; ++i) yh[i] = (yh[i] - mean_y) * r_y;
        }
      }
    }
    if (GATE == kFullGate) {
#pragma unroll
      for (int i = 0; i < 8; ++i) a[i] = 0.f;
      if (in) octet_floats(load_octet<TY>(row_at<TY>(p.gate.p, row, p.gate.row), oct), a);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        a[i] = gate_act(p.act, a[i]);
        slope[i] = p.beta * gate_slope(p.act, a[i]);
        a[i] *= p.beta;
      }
    }
    if (GATE == kOneGate && p.gate_kind == FLCE_GATE_TOKEN) {
      a[0] = gate_act(p.act, one_element<TY>(p.gate.p, false, row * p.gate.row));
      slope[0] = p.beta * gate_slope(p.act, a[0]);
      a[0] *= p.beta;
    }
    // sums: g xh, [g], and with a post-norm q yh e, q yh xh, [q yh, q e, q, q xh]
    constexpr int K = POST ? (AFF ? 8 : 3) : (AFF ? 2 : 1);
    float v[K];
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float g = dz[i] * w_pre[i];
      v[0] = fmaf(g, xh[i], v[0]);
      e[i] = fmaf(r_h, g, e[i]);
      if (AFF) v[K - 1] += g;
      if (POST) {
        const float ai = GATE == kNoGate ? p.beta : GATE == kOneGate ? a[0] : a[i];
        const float q = ai * w_post[i], qy = q * yh[i];
        v[1] = fmaf(qy, e[i], v[1]);
        v[2] = fmaf(qy, xh[i], v[2]);
        if (AFF) {
          v[3] += qy;
          v[4] = fmaf(q, e[i], v[4]);
          v[5] += q;
          v[6] = fmaf(q, xh[i], v[6]);
        }
      }
    }
    if (p.pre || POST) {
      sums.add(v);
      more.add(v);
    }
    const float m2 = r_h * v[0] * p.inv_h;
    const float m1 = AFF && layer ? r_h * v[K - 1] * p.inv_h : 0.f;
    float c1 = 0.f, c2 = 0.f;
    if (POST) {
      c2 = (v[1] - m2 * v[2] - (AFF ? m1 * v[3] : 0.f)) * p.inv_h;
      if (AFF && layer) c1 = (v[4] - m2 * v[6] - m1 * v[5]) * p.inv_h;
    }
    float one = 0.f;
    float dt[8], dg[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      dt[i] = fmaf(-m2, xh[i], e[i]) - m1;
      const float ai = GATE == kNoGate ? p.beta : GATE == kOneGate ? a[0] : a[i];
      const float du = ai * dt[i];
      if (GATE != kNoGate) {
        const float u = POST ? fmaf(yh[i], w_post[i], AFF ? b_post[i] : 0.f) : yh[i];
        if (GATE == kOneGate)
          one = fmaf(u, in ? dt[i] : 0.f, one);
        else
          dg[i] = slope[i] * u * dt[i];
        if (GATE == kChannelGate) s_gate[i] += dg[i];
      }
      s_wpre[i] = fmaf(dz[i], xh[i], s_wpre[i]);
      if (AFF) s_bpre[i] += dz[i];
      if (POST) {
        s_wpost[i] = fmaf(du, yh[i], s_wpost[i]);
        if (AFF) s_bpost[i] += du;
      }
      e[i] = POST ? r_y * (fmaf(-c2, yh[i], du * w_post[i]) - c1) : du;  // dy
      dt[i] *= p.alpha;                                                  // dh
    }
    if (in) {
      store_octet<TY>(row_at<TY>(p.dy.p, row, p.dy.row), oct, e);
      if (p.dh.p) store_octet<TH>(row_at<TH>(p.dh.p, row, p.dh.row), oct, dt);
      if (GATE == kFullGate) store_octet<TY>(row_at<TY>(p.dgate.p, row, p.dgate.row), oct, dg);
    }
    if (GATE == kOneGate) {
      if (p.gate_kind == FLCE_GATE_TOKEN) {
        float t[1] = {one};
        sums.add(t);
        more.add(t);
        if (in_cta == 0 && rank == 0) store_element(TY{}, p.dgate.p, row * p.dgate.row, slope[0] * t[0]);
      } else {
        s_gate[0] = fmaf(slope[0], one, s_gate[0]);
      }
    }
  }

  auto put = [&](float* part, const float (&s)[8]) {
    if (!part || !in) return;
    store_octet<float>(part + unit * p.H, oct, s);
  };
  put(p.part[0], s_wpre);
  if (AFF) put(p.part[1], s_bpre);
  if (POST) put(p.part[2], s_wpost);
  if (POST && AFF) put(p.part[3], s_bpost);
  if (GATE == kChannelGate) put(p.part[4], s_gate);
  if (GATE == kOneGate && p.part[4]) {
    float t[1] = {s_gate[0]};
    sums.add(t);
    more.add(t);
    if (in_cta == 0 && rank == 0) p.part[4][unit] = t[0];
  }
  if (p.cluster > 1) cluster_sync();  // no CTA leaves while another writes to its slots
}

template <class TY, class TH, bool POST, bool AFF, int GATE>
cudaError_t launch_bwd(const NormParams& p, int64_t parts, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(static_cast<unsigned>(parts / p.groups * p.cluster));
  cfg.blockDim = dim3(static_cast<unsigned>(32 * p.warps * p.groups));
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(p.cluster);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, resnorm_bwd_kernel<TY, TH, POST, AFF, GATE>, p);
}

template <class TY, class TH, bool POST, bool AFF>
cudaError_t launch_bwd_gate(const NormParams& p, int64_t parts, cudaStream_t s) {
  switch (p.gate_kind) {
    case FLCE_GATE_NONE:
      return launch_bwd<TY, TH, POST, AFF, kNoGate>(p, parts, s);
    case FLCE_GATE_CHANNEL:
      return launch_bwd<TY, TH, POST, AFF, kChannelGate>(p, parts, s);
    case FLCE_GATE_FULL:
      return launch_bwd<TY, TH, POST, AFF, kFullGate>(p, parts, s);
    default:
      return launch_bwd<TY, TH, POST, AFF, kOneGate>(p, parts, s);
  }
}

template <class TY, class TH>
cudaError_t launch_bwd_types(const NormParams& p, int64_t parts, cudaStream_t s) {
  const bool aff = p.layer || p.b_post || p.part[1] || p.part[3];
  if (p.post)
    return aff ? launch_bwd_gate<TY, TH, true, true>(p, parts, s)
               : launch_bwd_gate<TY, TH, true, false>(p, parts, s);
  return aff ? launch_bwd_gate<TY, TH, false, true>(p, parts, s)
             : launch_bwd_gate<TY, TH, false, false>(p, parts, s);
}

}  // namespace flce
