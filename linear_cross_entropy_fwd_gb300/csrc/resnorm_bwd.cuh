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

// Rows that a group takes at a time: two share the exchange of their sums, where the
// registers hold two (8192 x 4096 in bf16 with both norms: 75 us with one).
template <class TY, class TH, bool POST, int GATE>
constexpr int kBwdFit = ring_stages(kBwdPieces<TY, TH, POST, GATE>, kBwdThreads, kSmemPerSm, 6);
template <class TY, class TH, bool POST, bool AFF, int GATE>
constexpr int kBwdRows = POST && !AFF && (GATE == kNoGate || GATE == kChannelGate) &&
                                 kBwdFit<TY, TH, POST, GATE> >= 4
                             ? 2
                             : 1;
template <class TY, class TH, bool POST, bool AFF, int GATE>
constexpr int kBwdStages = kBwdFit<TY, TH, POST, GATE> / kBwdRows<TY, TH, POST, AFF, GATE> *
                           kBwdRows<TY, TH, POST, AFF, GATE>;

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
  grid_launch_dependents();  // the sums' CTAs take the SMs that this launch's leave
  const int in_cta = sums.warp * 32 + lane;
  const int oct = rank * p.octets + in_cta;
  const bool in = in_cta < p.octets && oct < p.H / 8;
  const bool pfp = p.params_fp32, layer = p.layer;
  constexpr bool kReadsY = POST || GATE != kNoGate;
  // a is the same in every row, so that it and the weight multiply the sums, not the rows
  constexpr bool kFixed = GATE == kNoGate || GATE == kChannelGate;

  const int64_t unit = static_cast<int64_t>(blockIdx.x / p.cluster) * p.groups + group;
  const int64_t units = static_cast<int64_t>(gridDim.x / p.cluster) * p.groups;
  const uint32_t step = blockDim.x * 16;
  const uint32_t ring = smem_addr(ring_raw) + threadIdx.x * 16;
  constexpr int R = kBwdRows<TY, TH, POST, AFF, GATE>;
  constexpr int kStages = kBwdStages<TY, TH, POST, AFF, GATE>;
  const uint32_t stage = step * kBwdPieces<TY, TH, POST, GATE>, end = kStages * stage;
  const uint32_t at_h = kPieces<TY> * step, at_dh = at_h + kPieces<TH> * step;
  const uint32_t at_y = at_dh + kPieces<TH> * step, at_gate = at_y + kPieces<TY> * step;
  int64_t ahead = unit;
  Walk<TY> dz_in(p.dz.p, p.dz.row, unit, oct), y_in(p.y.p, p.y.row, unit, oct);
  Walk<TH> h_in(p.h_out.p, p.h_out.row, unit, oct);
  Walk<TH> dh_in(p.dh_out.p, p.dh_out.row, unit, oct);
  Walk<TY> gate_in(p.gate.p, p.gate.row, unit, oct);
  auto fetch = [&](uint32_t s) {
    if (in && ahead < p.N) {
      const uint32_t at = ring + s;
      if (p.pre) {
        copy_octet<TY>(at, step, dz_in.at);
        copy_octet<TH>(at + at_h, step, h_in.at);
      }
      if (p.dh_out.p) copy_octet<TH>(at + at_dh, step, dh_in.at);
      if (kReadsY) copy_octet<TY>(at + at_y, step, y_in.at);
      if (GATE == kFullGate) copy_octet<TY>(at + at_gate, step, gate_in.at);
      ahead += units;
      dz_in.at += p.dz.step;
      h_in.at += p.h_out.step;
      dh_in.at += p.dh_out.step;
      if (kReadsY) y_in.at += p.y.step;
      if (GATE == kFullGate) gate_in.at += p.gate.step;
    }
    copies_commit();
  };
  uint32_t s_in = 0, s_out = 0;
  for (; s_in < end - R * stage; s_in += stage) fetch(s_in);
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
  Row next[R];
#pragma unroll
  for (int q = 0; q < R; ++q) next[q] = read_row(unit + q * units);

  auto gate_of_channel = [&]() {  // act(gate), 1 without one
    if (GATE != kChannelGate) return same_oct(1.f);
    return gate_act_oct(p.act, param_octet<TY>(p.gate.p, pfp, oct, 1.f));
  };
  // w_post: times beta a where that is fixed
  Oct w_pre = zero_oct(), w_post = zero_oct(), b_post = zero_oct();
  if (in) {
    w_pre = param_octet<TY>(p.w_pre, pfp, oct, 1.f);
    w_post = param_octet<TY>(POST ? p.w_post : nullptr, pfp, oct, 1.f);
    if (kFixed) {
      scale_oct(w_post, gate_of_channel());
      scale_oct(w_post, p.beta);
    } else if (POST && AFF) {
      b_post = param_octet<TY>(p.b_post, pfp, oct, 0.f);
    }
  }
  float scalar = 0.f;
  if (GATE == kOneGate && p.gate_kind == FLCE_GATE_SCALAR) scalar = one_element<TY>(p.gate.p, pfp, 0);

  // Sums over tokens: dz xh, dz, and with a fixed gate yh dt, dt; else yh du, du.
  Oct s_pre = zero_oct(), s_bpre = zero_oct(), s_post = zero_oct(), s_bpost = zero_oct();
  float s_one = 0.f;
  Walk<TY> dy(p.dy.p, p.dy.row, unit, oct), dgate(p.dgate.p, p.dgate.row, unit, oct);
  Walk<TH> dh(p.dh.p, p.dh.row, unit, oct);
  for (int64_t row = unit; row < p.N; row += R * units) {
#pragma unroll
    for (int q = 0; q < R; ++q) fetch(s_in + q * stage);
    s_in = s_in + R * stage == end ? 0 : s_in + R * stage;
    Row t[R];
    bool there[R];  // this thread has an octet of the row
#pragma unroll
    for (int q = 0; q < R; ++q) {
      t[q] = next[q];
      next[q] = read_row(row + (R + q) * units);
      there[q] = in && (q == 0 || row + q * units < p.N);
    }
    copies_wait<kStages - R>();

    Oct dz, xh, e, yh, a = zero_oct(), slope = zero_oct();
    float one_a = 0.f, one_slope = 0.f;
    // beta act(gate) and its slope
    auto act_of = [&](float g, float& value, float& gradient) {
      g = gate_act(p.act, g);
      gradient = p.beta * gate_slope(p.act, g);
      value = p.beta * g;
    };
    // beta a, and beta a w_post
    auto gate_at = [&](int i) { return GATE == kOneGate ? pair(one_a) : a.p[i]; };
    auto weight = [&](int i) { return kFixed ? w_post.p[i] : mul2(gate_at(i), w_post.p[i]); };
    // row q's dz, xh, e = dh' + r g and yh; a second time where two rows are in hand, which
    // takes fewer registers than keeping them
    auto read = [&](int q) {
      const uint32_t at = ring + s_out + q * stage;
      dz = xh = e = yh = a = zero_oct();
      if (there[q]) {
        if (p.pre) {
          dz = shared_octet(TY{}, at, step);
          xh = shared_octet(TH{}, at + at_h, step);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            xh.p[i] = mul2(AFF ? plus2(xh.p[i], pair(-t[q].mean_h)) : xh.p[i], pair(t[q].r_h));
        }
        if (p.dh_out.p) e = shared_octet(TH{}, at + at_dh, step);
        if (kReadsY) yh = shared_octet(TY{}, at + at_y, step);
        if (POST) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            yh.p[i] = mul2(AFF ? plus2(yh.p[i], pair(-t[q].mean_y)) : yh.p[i], pair(t[q].r_y));
        }
        if (GATE == kFullGate) a = shared_octet(TY{}, at + at_gate, step);
      }
      if (GATE == kFullGate) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          act_of(a.p[i].x, a.p[i].x, slope.p[i].x);
          act_of(a.p[i].y, a.p[i].y, slope.p[i].y);
        }
      }
      if (GATE == kOneGate)
        act_of(p.gate_kind == FLCE_GATE_TOKEN ? t[q].gate : scalar, one_a, one_slope);
    };
    // sums of a row: g xh, [g], and with a post-norm q yh e, q yh xh, [q yh, q e, q, q xh]
    constexpr int K = POST ? (AFF ? 8 : 4) : (AFF ? 2 : 1);
    float s[R * K];
#pragma unroll
    for (int q = 0; q < R; ++q) {
      read(q);
      float2 v[K];
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] = pair(0.f);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 g = mul2(dz.p[i], w_pre.p[i]);
        v[0] = mad2(g, xh.p[i], v[0]);
        e.p[i] = mad2(pair(t[q].r_h), g, e.p[i]);
        if (AFF) v[K - 1] = plus2(v[K - 1], g);
        if (POST) {
          const float2 w = weight(i), wy = mul2(w, yh.p[i]);
          v[1] = mad2(wy, e.p[i], v[1]);
          v[2] = mad2(wy, xh.p[i], v[2]);
          if (AFF) {
            v[3] = plus2(v[3], wy);
            v[4] = mad2(w, e.p[i], v[4]);
            v[5] = plus2(v[5], w);
            v[6] = mad2(w, xh.p[i], v[6]);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < K; ++k) s[q * K + k] = v[k].x + v[k].y;
    }
    if (p.pre || POST) {
      sums.add(s);
      more.add(s);
    }

#pragma unroll
    for (int q = 0; q < R; ++q) {
      const float r_h = t[q].r_h, r_y = t[q].r_y;
      const float m2 = r_h * s[q * K] * p.inv_h;
      const float m1 = AFF && layer ? r_h * s[q * K + K - 1] * p.inv_h : 0.f;
      float c1 = 0.f, c2 = 0.f;
      if (POST) {
        const float* v = &s[q * K];
        c2 = r_y * p.inv_h * (v[1] - m2 * v[2] - (AFF ? m1 * v[3] : 0.f));
        if (AFF && layer) c1 = r_y * p.inv_h * (v[4] - m2 * v[6] - m1 * v[5]);
      }
      if (R > 1) read(q);
      float2 one = pair(0.f);
      Oct dg;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (R > 1) e.p[i] = mad2(pair(r_h), mul2(dz.p[i], w_pre.p[i]), e.p[i]);
        float2 dt = mad2(pair(-m2), xh.p[i], e.p[i]);
        if (AFF) dt = plus2(dt, pair(-m1));
        s_pre.p[i] = mad2(dz.p[i], xh.p[i], s_pre.p[i]);
        if (AFF) s_bpre.p[i] = plus2(s_bpre.p[i], dz.p[i]);
        float2 gy = mul2(weight(i), dt);
        if (kFixed) {
          if (kReadsY) s_post.p[i] = mad2(yh.p[i], dt, s_post.p[i]);
          if (POST && AFF) s_bpost.p[i] = plus2(s_bpost.p[i], dt);
        } else {
          const float2 du = mul2(gate_at(i), dt);
          const float2 u = POST ? (AFF ? mad2(yh.p[i], w_post.p[i], b_post.p[i])
                                       : mul2(yh.p[i], w_post.p[i]))
                                : yh.p[i];
          if (GATE == kOneGate)
            one = mad2(u, in ? dt : pair(0.f), one);
          else
            dg.p[i] = mul2(mul2(slope.p[i], u), dt);
          if (POST) s_post.p[i] = mad2(yh.p[i], du, s_post.p[i]);
          if (POST && AFF) s_bpost.p[i] = plus2(s_bpost.p[i], du);
        }
        if (POST) {
          gy = mad2(pair(-c2), yh.p[i], mul2(pair(r_y), gy));
          if (AFF) gy = plus2(gy, pair(-c1));
        }
        e.p[i] = gy;                        // dy
        xh.p[i] = mul2(pair(p.alpha), dt);  // dh
      }
      if (there[q]) {
        dy.put(to_octet(TY{}, e));
        if (p.dh.p) dh.put(to_octet(TH{}, xh));
        if (GATE == kFullGate) dgate.put(to_octet(TY{}, dg));
      }
      dy.at += p.dy.step;
      dh.at += p.dh.step;
      if (GATE == kFullGate) dgate.at += p.dgate.step;
      if (GATE == kOneGate) {
        if (p.gate_kind == FLCE_GATE_TOKEN) {
          float d[1] = {one.x + one.y};
          sums.add(d);
          more.add(d);
          if (in_cta == 0 && rank == 0)
            store_element(TY{}, p.dgate.p, row * p.dgate.row, one_slope * d[0]);
        } else {
          s_one = fmaf(one_slope, one.x + one.y, s_one);
        }
      }
    }
    s_out = s_out + R * stage == end ? 0 : s_out + R * stage;
  }

  auto put = [&](float* part, const Oct& o) {
    if (part && in) store_octet<float>(part + unit * p.H, oct, o);
  };
  put(p.part[0], s_pre);
  if (AFF) put(p.part[1], s_bpre);
  if (kFixed && kReadsY && in) {
    Oct a = gate_of_channel();
    if (GATE == kChannelGate) {
      // dgate = slope (w_post sum yh dt + b_post sum dt)
      Oct f = param_octet<TY>(POST ? p.w_post : nullptr, pfp, oct, 1.f);
      scale_oct(f, s_post);
      if (POST && AFF) {
        b_post = param_octet<TY>(p.b_post, pfp, oct, 0.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) f.p[i] = mad2(b_post.p[i], s_bpost.p[i], f.p[i]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        f.p[i] = mul2(f.p[i], make_float2(p.beta * gate_slope(p.act, a.p[i].x),
                                          p.beta * gate_slope(p.act, a.p[i].y)));
      put(p.part[4], f);
    }
    scale_oct(a, p.beta);
    scale_oct(s_post, a);
    scale_oct(s_bpost, a);
  }
  if (POST) put(p.part[2], s_post);
  if (POST && AFF) put(p.part[3], s_bpost);
  if (GATE == kOneGate && p.part[4]) {
    float d[1] = {s_one};
    sums.add(d);
    more.add(d);
    if (in_cta == 0 && rank == 0) p.part[4][unit] = d[0];
  }
  if (p.cluster > 1) cluster_sync();  // no CTA leaves while another writes to its slots
}

template <class TY, class TH, bool POST, bool AFF, int GATE>
cudaError_t launch_bwd(NormParams p, int64_t parts, cudaStream_t s) {
  static SmemLimit limit;
  const int threads = 32 * p.warps * p.groups;
  const int ring = threads * 16 * kBwdPieces<TY, TH, POST, GATE> *
                   kBwdStages<TY, TH, POST, AFF, GATE>;
  const auto kernel = resnorm_bwd_kernel<TY, TH, POST, AFF, GATE>;
  const cudaError_t e = limit.raise(kernel, kSmemPerSm);
  if (e != cudaSuccess) return e;
  set_steps(p, parts, Elem<TY>::kBytes, Elem<TH>::kBytes);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(static_cast<unsigned>(parts / p.groups * p.cluster));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(ring);
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
