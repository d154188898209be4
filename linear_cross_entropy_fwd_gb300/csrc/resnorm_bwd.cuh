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

// 16-byte pieces of a stage of the ring, per thread: dz, h', dh' and, where they are read, y
// and a gate per element.
template <class TY, class TH, bool POST, int GATE>
constexpr int kBwdPieces =
    kPieces<TY> + 2 * kPieces<TH> + (POST || GATE != kNoGate ? kPieces<TY> : 0) +
    (GATE == kFullGate ? kPieces<TY> : 0);

// AFF: a mean or a bias is wanted.
template <class TY, class TH, bool POST, bool AFF, int GATE>
__global__ void __launch_bounds__(kBwdThreads, 1)
    resnorm_bwd_kernel(const __grid_constant__ NormParams p) {
  __shared__ float slots[kMaxRowWarps][2][kMaxSums][kMaxRowWarps];
  __shared__ float cluster_slots[2][4][kMaxSums];
  extern __shared__ __align__(16) uint8_t ring_raw[];
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
  constexpr bool kReadsY = POST || GATE != kNoGate;
  // a is the same in every row, so that it and the weight multiply the sums, not the rows
  constexpr bool kFixed = GATE == kNoGate || GATE == kChannelGate;

  const uint32_t step = blockDim.x * 16;
  const uint32_t ring = smem_addr(ring_raw) + threadIdx.x * 16;
  const uint32_t stage = step * kBwdPieces<TY, TH, POST, GATE>;
  const uint32_t at_h = kPieces<TY> * step, at_dh = at_h + kPieces<TH> * step;
  const uint32_t at_y = at_dh + kPieces<TH> * step, at_gate = at_y + kPieces<TY> * step;
  auto fetch = [&](int64_t row, int s) {
    if (in && row < p.N) {
      const uint32_t at = ring + s * stage;
      if (p.pre) {
        copy_octet<TY>(at, step, row_at<TY>(p.dz.p, row, p.dz.row), oct);
        copy_octet<TH>(at + at_h, step, row_at<TH>(p.h_out.p, row, p.h_out.row), oct);
      }
      if (p.dh_out.p)
        copy_octet<TH>(at + at_dh, step, row_at<TH>(p.dh_out.p, row, p.dh_out.row), oct);
      if (kReadsY) copy_octet<TY>(at + at_y, step, row_at<TY>(p.y.p, row, p.y.row), oct);
      if (GATE == kFullGate)
        copy_octet<TY>(at + at_gate, step, row_at<TY>(p.gate.p, row, p.gate.row), oct);
    }
    copies_commit();
  };
  // a row's statistics, and its gate of one value, one row ahead
  struct Row {
    float mean_y, r_y, mean_h, r_h, gate;
  };
  auto read_row = [&](int64_t row) {
    Row t{0.f, 1.f, 0.f, 0.f, 0.f};
    if (row >= p.N) return t;
    if (POST) {
      if (AFF) t.mean_y = p.stats[row];
      t.r_y = p.stats[p.N + row];
    }
    if (p.pre) {
      if (AFF) t.mean_h = p.stats[2 * p.N + row];
      t.r_h = p.stats[3 * p.N + row];
    }
    if (GATE == kOneGate && p.gate_kind == FLCE_GATE_TOKEN)
      t.gate = one_element<TY>(p.gate.p, false, row * p.gate.row);
    return t;
  };

  float w_pre[8], w_post[8], b_post[8];  // w_post: times beta a where that is fixed
#pragma unroll
  for (int i = 0; i < 8; ++i) w_pre[i] = w_post[i] = b_post[i] = 0.f;
  auto gate_of_channel = [&](float (&a)[8]) {  // act(gate), 1 without one
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = 1.f;
    if (GATE == kChannelGate) {
      param_octet<TY>(p.gate.p, pfp, oct, 1.f, a);
#pragma unroll
      for (int i = 0; i < 8; ++i) a[i] = gate_act(p.act, a[i]);
    }
  };
  if (in) {
    param_octet<TY>(p.w_pre, pfp, oct, 1.f, w_pre);
    param_octet<TY>(POST ? p.w_post : nullptr, pfp, oct, 1.f, w_post);
    if (kFixed) {
      float a[8];
      gate_of_channel(a);
#pragma unroll
      for (int i = 0; i < 8; ++i) w_post[i] *= p.beta * a[i];
    } else if (POST && AFF) {
      param_octet<TY>(p.b_post, pfp, oct, 0.f, b_post);
    }
  }
  float scalar = 0.f;
  if (GATE == kOneGate && p.gate_kind == FLCE_GATE_SCALAR) scalar = one_element<TY>(p.gate.p, pfp, 0);

  // Sums over tokens: dz xh, dz, and with a fixed gate yh dt, dt; else yh du, du.
  float s_pre[8], s_bpre[8], s_post[8], s_bpost[8], s_one = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s_pre[i] = s_bpre[i] = s_post[i] = s_bpost[i] = 0.f;

  const int64_t unit = static_cast<int64_t>(blockIdx.x / p.cluster) * p.groups + group;
  const int64_t units = static_cast<int64_t>(gridDim.x / p.cluster) * p.groups;
  int s_in = 0, s_out = 0;
  for (; s_in < p.stages - 1; ++s_in) fetch(unit + s_in * units, s_in);
  Row next = read_row(unit);
  for (int64_t row = unit; row < p.N; row += units) {
    fetch(row + (p.stages - 1) * units, s_in);
    s_in = s_in + 1 == p.stages ? 0 : s_in + 1;
    const Row t = next;
    next = read_row(row + units);
    copies_wait(p.stages - 1);
    const uint32_t at = ring + s_out * stage;
    s_out = s_out + 1 == p.stages ? 0 : s_out + 1;

    float dz[8], xh[8], e[8], yh[8], a[8], slope[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) dz[i] = xh[i] = e[i] = yh[i] = a[i] = slope[i] = 0.f;
    if (in) {
      if (p.pre) {
        shared_octet(TY{}, at, step, dz);
        shared_octet(TH{}, at + at_h, step, xh);
#pragma unroll
        for (int i = 0; i < 8; ++i) xh[i] = AFF ? (xh[i] - t.mean_h) * t.r_h : xh[i] * t.r_h;
      }
      if (p.dh_out.p) shared_octet(TH{}, at + at_dh, step, e);
      if (kReadsY) shared_octet(TY{}, at + at_y, step, yh);
      if (POST) {
#pragma unroll
        for (int i = 0; i < 8; ++i) yh[i] = AFF ? (yh[i] - t.mean_y) * t.r_y : yh[i] * t.r_y;
      }
      if (GATE == kFullGate) shared_octet(TY{}, at + at_gate, step, a);
    }
    // beta act(gate) and its slope
    if (GATE == kFullGate || GATE == kOneGate) {
#pragma unroll
      for (int i = 0; i < (GATE == kOneGate ? 1 : 8); ++i) {
        if (GATE == kOneGate) a[i] = p.gate_kind == FLCE_GATE_TOKEN ? t.gate : scalar;
        a[i] = gate_act(p.act, a[i]);
        slope[i] = p.beta * gate_slope(p.act, a[i]);
        a[i] *= p.beta;
      }
    }
    // beta a w_post of element i
    auto weight = [&](int i) {
      return kFixed ? w_post[i] : (GATE == kOneGate ? a[0] : a[i]) * w_post[i];
    };

    // sums: g xh, [g], and with a post-norm q yh e, q yh xh, [q yh, q e, q, q xh]
    constexpr int K = POST ? (AFF ? 8 : 4) : (AFF ? 2 : 1);
    float v[K];
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float g = dz[i] * w_pre[i];
      v[0] = fmaf(g, xh[i], v[0]);
      e[i] = fmaf(t.r_h, g, e[i]);
      if (AFF) v[K - 1] += g;
      if (POST) {
        const float q = weight(i), qy = q * yh[i];
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
    const float m2 = t.r_h * v[0] * p.inv_h;
    const float m1 = AFF && layer ? t.r_h * v[K - 1] * p.inv_h : 0.f;
    float c1 = 0.f, c2 = 0.f;
    if (POST) {
      c2 = (v[1] - m2 * v[2] - (AFF ? m1 * v[3] : 0.f)) * p.inv_h;
      if (AFF && layer) c1 = (v[4] - m2 * v[6] - m1 * v[5]) * p.inv_h;
    }
    float one = 0.f, dg[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float dt = fmaf(-m2, xh[i], e[i]);
      if (AFF) dt -= m1;
      s_pre[i] = fmaf(dz[i], xh[i], s_pre[i]);
      if (AFF) s_bpre[i] += dz[i];
      const float gy = weight(i) * dt;
      if (kFixed) {
        if (kReadsY) s_post[i] = fmaf(yh[i], dt, s_post[i]);
        if (POST && AFF) s_bpost[i] += dt;
      } else {
        const float du = (GATE == kOneGate ? a[0] : a[i]) * dt;
        const float u = POST ? fmaf(yh[i], w_post[i], AFF ? b_post[i] : 0.f) : yh[i];
        if (GATE == kOneGate)
          one = fmaf(u, in ? dt : 0.f, one);
        else
          dg[i] = slope[i] * u * dt;
        if (POST) s_post[i] = fmaf(yh[i], du, s_post[i]);
        if (POST && AFF) s_bpost[i] += du;
      }
      xh[i] = p.alpha * dt;                                           // dh
      e[i] = POST ? t.r_y * (fmaf(-c2, yh[i], gy) - (AFF ? c1 : 0.f)) : gy;  // dy
    }
    if (in) {
      store_octet<TY>(row_at<TY>(p.dy.p, row, p.dy.row), oct, e);
      if (p.dh.p) store_octet<TH>(row_at<TH>(p.dh.p, row, p.dh.row), oct, xh);
      if (GATE == kFullGate) store_octet<TY>(row_at<TY>(p.dgate.p, row, p.dgate.row), oct, dg);
    }
    if (GATE == kOneGate) {
      if (p.gate_kind == FLCE_GATE_TOKEN) {
        float s[1] = {one};
        sums.add(s);
        more.add(s);
        if (in_cta == 0 && rank == 0)
          store_element(TY{}, p.dgate.p, row * p.dgate.row, slope[0] * s[0]);
      } else {
        s_one = fmaf(slope[0], one, s_one);
      }
    }
  }

  auto put = [&](float* part, const float (&s)[8]) {
    if (part && in) store_octet<float>(part + unit * p.H, oct, s);
  };
  put(p.part[0], s_pre);
  if (AFF) put(p.part[1], s_bpre);
  if (kFixed && kReadsY && in) {
    float a[8], f[8];
    gate_of_channel(a);
    if (GATE == kChannelGate) {
      // dgate = slope (w_post sum yh dt + b_post sum dt)
      param_octet<TY>(POST ? p.w_post : nullptr, pfp, oct, 1.f, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] *= s_post[i];
      if (POST && AFF) {
        param_octet<TY>(p.b_post, pfp, oct, 0.f, b_post);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = fmaf(b_post[i], s_bpost[i], f[i]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] *= p.beta * gate_slope(p.act, a[i]);
      put(p.part[4], f);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      s_post[i] *= p.beta * a[i];
      s_bpost[i] *= p.beta * a[i];
    }
  }
  if (POST) put(p.part[2], s_post);
  if (POST && AFF) put(p.part[3], s_bpost);
  if (GATE == kOneGate && p.part[4]) {
    float s[1] = {s_one};
    sums.add(s);
    more.add(s);
    if (in_cta == 0 && rank == 0) p.part[4][unit] = s[0];
  }
  if (p.cluster > 1) cluster_sync();  // no CTA leaves while another writes to its slots
}

template <class TY, class TH, bool POST, bool AFF, int GATE>
cudaError_t launch_bwd(NormParams p, int64_t parts, cudaStream_t s) {
  static SmemLimit limit;
  const int threads = 32 * p.warps * p.groups;
  const int stage = threads * 16 * kBwdPieces<TY, TH, POST, GATE>;
  p.stages = kSmemPerSm / stage < kMaxStages ? kSmemPerSm / stage : kMaxStages;
  const auto kernel = resnorm_bwd_kernel<TY, TH, POST, AFF, GATE>;
  const cudaError_t e = limit.raise(kernel, kSmemPerSm);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(static_cast<unsigned>(parts / p.groups * p.cluster));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(p.stages) * stage;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(p.cluster);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
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
