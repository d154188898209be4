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
// And behind the pieces, for each warp, the row's four statistics and its gate of one value:
// a load a row ahead would have to keep registers through the row, or is moved to where it is
// waited for (8192 x 4096 with gates per element 131 us, 54 of them waiting).
constexpr uint32_t kRowBytes = 32, kTailBytes = kRowBytes * kMaxRowWarps;

// Weights that wait in shared memory behind the ring instead of in registers: where a norm
// after the block and its means or biases need those for sums.
template <bool POST, bool AFF, int GATE>
constexpr int kBwdVectors = POST && AFF ? (GATE == kFullGate ? 3 : 2) : 0;
template <class TY, class TH, bool POST, bool AFF, int GATE>
constexpr int kBwdFit =
    ring_stages(kBwdPieces<TY, TH, POST, GATE>, kBwdThreads,
                kSmemPerSm - 4 * static_cast<int>(kTailBytes) -
                    kBwdVectors<POST, AFF, GATE> * kBwdThreads * 32,
                4);
template <class TY, class TH, bool POST, bool AFF, int GATE>
constexpr int kBwdRows = POST && !AFF && (GATE == kNoGate || GATE == kChannelGate) &&
                                 kBwdFit<TY, TH, POST, AFF, GATE> >= 4
                             ? 2
                             : 1;
template <class TY, class TH, bool POST, bool AFF, int GATE>
constexpr int kBwdStages = kBwdFit<TY, TH, POST, AFF, GATE> / kBwdRows<TY, TH, POST, AFF, GATE> *
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
  const uint32_t ring = smem_addr(ring_raw);
  const int mine = (p.octets < p.H / 8 - rank * p.octets ? p.octets : p.H / 8 - rank * p.octets);
  const Slot<TY> slot_y(threadIdx.x, lane, in_cta, mine);
  const Slot<TH> slot_h(threadIdx.x, lane, in_cta, mine);
  constexpr int R = kBwdRows<TY, TH, POST, AFF, GATE>;
  constexpr int kStages = kBwdStages<TY, TH, POST, AFF, GATE>;
  const uint32_t tail = step * kBwdPieces<TY, TH, POST, GATE>, stage = tail + kTailBytes;
  const uint32_t end = kStages * stage;
  const uint32_t my_tail = smem_addr(ring_raw) + tail + warp * kRowBytes;
  const uint32_t at_h = kPieces<TY> * step, at_dh = at_h + kPieces<TH> * step;
  const uint32_t at_y = at_dh + kPieces<TH> * step, at_gate = at_y + kPieces<TY> * step;
  constexpr bool kOwn = Slot<TY>::kOwn && Slot<TH>::kOwn;
  int64_t ahead = unit;
  Walk<TY> dz_in(p.dz.p, p.dz.row, unit, oct), y_in(p.y.p, p.y.row, unit, oct);
  Walk<TH> h_in(p.h_out.p, p.h_out.row, unit, oct);
  Walk<TH> dh_in(p.dh_out.p, p.dh_out.row, unit, oct);
  Walk<TY> gate_in(p.gate.p, p.gate.row, unit, oct);
  const bool token = GATE == kOneGate && p.gate_kind == FLCE_GATE_TOKEN;
  // address of a token's gate; its word, if all of that belongs to some token
  auto gate_of = [&](int64_t row) {
    return static_cast<const uint8_t*>(p.gate.p) + row * p.gate.row * Elem<TY>::kBytes;
  };
  auto fetch = [&](uint32_t s) {
    if (ahead < p.N) {
      const uint32_t at = ring + s;
      // one branch for all copies where a lane makes all of its own or none
      if (!kOwn || in) {
        if (p.pre) {
          slot_y.copy(at, dz_in.at, kOwn);
          slot_h.copy(at + at_h, h_in.at, kOwn);
        }
        if (p.dh_out.p) slot_h.copy(at + at_dh, dh_in.at, kOwn);
        if (kReadsY) slot_y.copy(at + at_y, y_in.at, kOwn);
        if (GATE == kFullGate) slot_y.copy(at + at_gate, gate_in.at, kOwn);
      }
      if (lane < 4) {
        if (lane < 2 ? POST : p.pre != 0)
          copy4(my_tail + s + 4 * lane, p.stats + lane * p.N + ahead);
      } else if (lane == 4 && token) {
        const uint8_t* g = gate_of(ahead);
        const uint8_t* word = g - (reinterpret_cast<uintptr_t>(g) & 3);
        if (Elem<TY>::kBytes == 4 || (word >= gate_of(0) && word + 2 <= gate_of(p.N - 1)))
          copy4(my_tail + s + 16, word);
        else  // the first or the last of a tensor that ends within a word
          st_shared4(my_tail + s + 16, static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(g))
                                           << (8 * (g - word)));
      }
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
  auto gate_of_channel = [&]() {  // act(gate), 1 without one
    if (GATE != kChannelGate) return same_oct(1.f);
    return gate_act_oct(p.act, param_octet<TY>(p.gate.p, pfp, oct, 1.f));
  };
  // w_post and b_post: times beta, and a where that is fixed
  constexpr bool kShared = kBwdVectors<POST, AFF, GATE> > 0;
  const uint32_t vectors = smem_addr(ring_raw) + end + in_cta * 16, plane = 32 * p.warps * 16;
  Oct w_pre = zero_oct(), w_post = zero_oct(), b_post = zero_oct();
  if (in) {
    w_pre = param_octet<TY>(p.w_pre, pfp, oct, 1.f);
    w_post = param_octet<TY>(POST ? p.w_post : nullptr, pfp, oct, 1.f);
    if (kFixed) scale_oct(w_post, gate_of_channel());
    scale_oct(w_post, p.beta);
    if (GATE == kFullGate && POST && AFF) {
      b_post = param_octet<TY>(p.b_post, pfp, oct, 0.f);
      scale_oct(b_post, p.beta);
    }
  }
  if (kShared) {
    if (group == 0) {
      put_shared(vectors, plane, w_pre);
      put_shared(vectors + 2 * plane, plane, w_post);
      if (GATE == kFullGate) put_shared(vectors + 4 * plane, plane, b_post);
    }
    __syncthreads();
  }
  auto pre_weight = [&]() { return kShared ? shared_oct(vectors, plane) : w_pre; };
  auto post_weight = [&]() {
    return kShared ? shared_oct(vectors + 2 * plane, plane) : w_post;
  };
  float scalar = 0.f;
  if (GATE == kOneGate && p.gate_kind == FLCE_GATE_SCALAR) scalar = one_element<TY>(p.gate.p, pfp, 0);

  // Sums over tokens: dz xh, dz, and yh du, du without the factor beta and a fixed gate's.
  Oct s_pre = zero_oct(), s_bpre = zero_oct(), s_post = zero_oct(), s_bpost = zero_oct();
  float s_one = 0.f;
  Walk<TY> dy(p.dy.p, p.dy.row, unit, oct), dgate(p.dgate.p, p.dgate.row, unit, oct);
  Walk<TH> dh(p.dh.p, p.dh.row, unit, oct);
  const GateSlope slope(p.act);
  for (int64_t row = unit; row < p.N; row += R * units) {
#pragma unroll
    for (int q = 0; q < R; ++q) fetch(s_in + q * stage);
    s_in = s_in + R * stage == end ? 0 : s_in + R * stage;
    bool there[R];  // this thread has an octet of the row
#pragma unroll
    for (int q = 0; q < R; ++q) there[q] = in && (q == 0 || row + q * units < p.N);
    copies_wait<kStages - R>();
    __syncwarp();  // lanes read what others copied

    Oct dz, xh, e, yh, a = zero_oct();
    float one = 0.f;  // act(gate) of gates with one value; `a` of those per element
    float mean_y, r_y, mean_h, r_h, rs_y[R], rs_h[R];
    // row q's dz, xh, dh' and yh; a second time where two rows are in hand, which takes
    // fewer registers than keeping them
    auto read = [&](int q, bool again) {
      const uint32_t at = ring + s_out + q * stage, row_at = my_tail + s_out + q * stage;
      if (again) {  // two rows are taken of RMS norms only
        mean_y = mean_h = 0.f;
        r_y = rs_y[q];
        r_h = rs_h[q];
      } else {
        const uint4 t = ld_shared16(row_at);
        mean_y = __uint_as_float(t.x);
        rs_y[q] = r_y = __uint_as_float(t.y);
        mean_h = __uint_as_float(t.z);
        rs_h[q] = r_h =
            p.pre && (q == 0 || row + q * units < p.N) ? __uint_as_float(t.w) : 0.f;
      }
      dz = xh = e = yh = a = zero_oct();
      if (there[q]) {
        if (p.pre) {
          dz = slot_y.read(at);
          xh = slot_h.read(at + at_h);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            xh.p[i] = mul2(AFF ? plus2(xh.p[i], pair(-mean_h)) : xh.p[i], pair(r_h));
        }
        if (p.dh_out.p) e = slot_h.read(at + at_dh);
        if (kReadsY) yh = slot_y.read(at + at_y);
        if (POST) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            yh.p[i] = mul2(AFF ? plus2(yh.p[i], pair(-mean_y)) : yh.p[i], pair(r_y));
        }
        if (GATE == kFullGate)
          a = gate_act_each(p.act, slot_y.read(at + at_gate));
      }
      if (GATE == kOneGate) {
        float g = scalar;
        if (token) {
          const uint32_t w = ld_shared4(row_at + 16);
          const bool upper = Elem<TY>::kBytes == 2 &&
                             (reinterpret_cast<uintptr_t>(gate_of(row + q * units)) & 2);
          g = element_value<TY>(upper ? w >> 16 : w, false);
        }
        one = gate_act(p.act, g);
      }
    };
    // Sums of a row: g xh, [g]; and with a post-norm or a gate of one value, with w for
    // beta [a] w_post: w yh e, w yh xh, [w yh], and for layer norms [w e, w, w xh].
    constexpr bool kSumsY = POST || GATE == kOneGate;
    constexpr int K = kSumsY ? (AFF ? 8 : 4) : (AFF ? 2 : 1);
    float s[R * K];
#pragma unroll
    for (int q = 0; q < R; ++q) {
      read(q, false);
      const Oct wp = pre_weight(), wq = post_weight();
      float2 v[K];
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] = pair(0.f);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 g = mul2(dz.p[i], wp.p[i]);
        v[0] = mad2(g, xh.p[i], v[0]);
        e.p[i] = mad2(pair(r_h), g, e.p[i]);
        if (AFF) v[K - 1] = plus2(v[K - 1], g);
        if (kSumsY) {
          const float2 w = GATE == kFullGate ? mul2(a.p[i], wq.p[i]) : wq.p[i];
          const float2 wy = mul2(w, yh.p[i]);
          v[1] = mad2(wy, e.p[i], v[1]);
          v[2] = mad2(wy, xh.p[i], v[2]);
          if (AFF) v[3] = plus2(v[3], wy);
          if (AFF && POST) {
            v[4] = mad2(w, e.p[i], v[4]);
            v[5] = plus2(v[5], w);
            v[6] = mad2(w, xh.p[i], v[6]);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < K; ++k) s[q * K + k] = v[k].x + v[k].y;
    }
    // (the exchanges also see to it that all lanes have read what later copies overwrite)
    if (p.pre || kSumsY) {
      sums.add(s);
      more.add(s);
    } else {
      __syncwarp();
    }

#pragma unroll
    for (int q = 0; q < R; ++q) {
      if (R > 1) {
        read(q, true);
        if (!kOwn && q == R - 1) __syncwarp();  // as above
      }
      const float m2 = r_h * s[q * K] * p.inv_h;
      const float m1 = AFF && layer ? r_h * s[q * K + K - 1] * p.inv_h : 0.f;
      // sum w yh dt: with a gate of one value its gradient, and dy's second mean
      float wyd = 0.f, c1 = 0.f, c2 = 0.f;
      if (kSumsY) wyd = s[q * K + 1] - m2 * s[q * K + 2] - (AFF ? m1 * s[q * K + 3] : 0.f);
      if (POST) {
        c2 = r_y * p.inv_h * wyd;
        if (AFF && layer)
          c1 = r_y * p.inv_h * (s[q * K + 4] - m2 * s[q * K + 6] - m1 * s[q * K + 5]);
      }
      if (GATE == kOneGate) {
        c1 *= one;
        c2 *= one;
      }
      const Oct wp = R > 1 ? pre_weight() : zero_oct(), wq = post_weight();
      const Oct bq = GATE == kFullGate && kShared
                         ? shared_oct(vectors + 4 * plane, plane)
                         : zero_oct();
      Oct dg = zero_oct();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (R > 1) e.p[i] = mad2(pair(r_h), mul2(dz.p[i], wp.p[i]), e.p[i]);
        float2 dt = mad2(pair(-m2), xh.p[i], e.p[i]);
        if (AFF) dt = plus2(dt, pair(-m1));
        s_pre.p[i] = mad2(dz.p[i], xh.p[i], s_pre.p[i]);
        if (AFF) s_bpre.p[i] = plus2(s_bpre.p[i], dz.p[i]);
        // du over beta, or beta a where that is fixed
        float2 du = dt;
        if (GATE == kOneGate) du = mul2(pair(one), dt);
        if (GATE == kFullGate) {
          du = mul2(a.p[i], dt);
          // beta u: w_post is times beta, and beta itself without a post-norm
          const float2 u = POST && AFF ? mad2(yh.p[i], wq.p[i], bq.p[i])
                                       : mul2(yh.p[i], wq.p[i]);
          dg.p[i] = mul2(mul2(slope(a.p[i]), u), dt);
        }
        if (POST || GATE == kChannelGate) s_post.p[i] = mad2(yh.p[i], du, s_post.p[i]);
        if (POST && AFF) s_bpost.p[i] = plus2(s_bpost.p[i], du);
        float2 gy = mul2(wq.p[i], du);
        if (POST) {
          gy = mad2(pair(-c2), yh.p[i], mul2(pair(r_y), gy));
          if (AFF) gy = plus2(gy, pair(-c1));
        }
        e.p[i] = gy;                        // dy
        a.p[i] = dt;
        xh.p[i] = mul2(pair(p.alpha), dt);  // dh
      }
      if (there[q]) {
        dy.put(to_octet(TY{}, e), p.wide);
        if (p.dh.p) dh.put(to_octet(TH{}, xh), p.wide);
        if (GATE == kFullGate) dgate.put(to_octet(TY{}, dg), p.wide);
      }
      dy.at += p.dy.step;
      dh.at += p.dh.step;
      if (GATE == kFullGate) dgate.at += p.dgate.step;
      if (GATE == kOneGate) {
        if (POST && p.b_post) {  // u has a part beside w yh
          float d[1] = {0.f};
          if (there[q]) {
            Oct b = param_octet<TY>(p.b_post, pfp, oct, 0.f);
            scale_oct(b, a);
            d[0] = p.beta * sum_oct(b);
          }
          sums.add(d);
          more.add(d);
          wyd += d[0];
        }
        wyd *= gate_slope(p.act, one);
        if (p.gate_kind == FLCE_GATE_SCALAR)
          s_one += wyd;
        else if (in_cta == 0 && rank == 0)
          store_element(TY{}, p.dgate.p, (row + q * units) * p.dgate.row, wyd);
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
    scale_oct(s_post, a);
    scale_oct(s_bpost, a);
  }
  scale_oct(s_post, p.beta);
  scale_oct(s_bpost, p.beta);
  if (POST) put(p.part[2], s_post);
  if (POST && AFF) put(p.part[3], s_bpost);
  if (GATE == kOneGate && p.part[4] && in_cta == 0 && rank == 0) p.part[4][unit] = s_one;
  if (p.cluster > 1) cluster_sync();  // no CTA leaves while another writes to its slots
}

template <class TY, class TH, bool POST, bool AFF, int GATE>
cudaError_t launch_bwd(NormParams p, int64_t parts, cudaStream_t s) {
  static SmemLimit limit;
  const int threads = 32 * p.warps * p.groups;
  const int vectors = kBwdVectors<POST, AFF, GATE> * 32 * p.warps * 32;
  const int ring = (threads * 16 * kBwdPieces<TY, TH, POST, GATE> + static_cast<int>(kTailBytes)) *
                   kBwdStages<TY, TH, POST, AFF, GATE>;
  const auto kernel = resnorm_bwd_kernel<TY, TH, POST, AFF, GATE>;
  const cudaError_t e = limit.raise(kernel, kSmemPerSm);
  if (e != cudaSuccess) return e;
  set_steps(p, parts, Elem<TY>::kBytes, Elem<TH>::kBytes);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(static_cast<unsigned>(parts / p.groups * p.cluster));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(ring + vectors);
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
