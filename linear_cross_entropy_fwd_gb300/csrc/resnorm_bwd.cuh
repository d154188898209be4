// resnorm_bwd.cuh -- the residual join's backward pass (resnorm.h has the formulas); one
// translation unit per pair of types includes it.
//
// Bound by memory where rows share what goes on around them: dz, dh', h' (and y) are read
// once, dh and dy written once.  8192 x 4096 in bf16: 57 us with a norm before the next block
// (5 streams, 5.9 TB/s), 73 us with one on both sides (6, 5.5 TB/s); 65536 x 4096 390 us (6.9
// TB/s) and 515 (6.3).  Means and biases on both sides make the instructions the bound: 89 us.
//
// A thread has the same NV octets of every row that its warps take, so that the sums over
// tokens stay in its registers until the end; the CTA's groups of warps add theirs in shared
// memory, one fp32 row for each CTA is left, and a second kernel adds those in a fixed order
// (without the step between, 65536 x 256: 63 us, 18 of them in the second kernel; 37 with it).
// One octet a thread, 4096 elements a CTA, is what 5 such sums leave room for, two what 2 or 3
// do; longer rows are shared by the CTAs of a cluster, at an exchange of 1 us more per row.
//
// The two norms' sums would follow one another (the post-norm's need dt, dt needs the
// pre-norm's).  But dt is linear in them: with e = dh' + r g and q = beta a w_post,
//   dt = e - r m1 - r m2 xh,   sum gy yh = sum q yh e - r m1 sum q yh - r m2 sum q yh xh
// (and the same without yh), so all sums of a row are taken together, one exchange per row.
#pragma once
#include <atomic>

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

// And behind the pieces, for each warp, the row's four statistics and its gate of one value:
// a load a row ahead would have to keep registers through the row, or is moved to where it is
// waited for (8192 x 4096 with gates per element: 131 us, 54 of them waiting; 90 now).
constexpr uint32_t kRowBytes = 32, kTailBytes = kRowBytes * kMaxRowWarps;

// What the launch and the kernel agree on, for NV octets a thread.
template <class TY, class TH, bool POST, bool AFF, int GATE, int NV>
struct BwdShape {
  static constexpr int kPiecesRow = NV * kBwdPieces<TY, TH, POST, GATE>;
  // Rows that a group takes at a time: two share the exchange of their sums, where the
  // registers hold two (8192 x 4096 in bf16 with both norms: 79 us with one, 71 with two).
  // With means or biases a second row takes longer to read again than it saves: 99 us, 89.
  static constexpr bool kTwoRows = NV == 1 && Elem<TH>::kBytes + Elem<TY>::kBytes <= 6 && POST &&
                                   !AFF && (GATE == kNoGate || GATE == kChannelGate);
  // Weights that wait in shared memory behind the ring instead of in registers: where a norm
  // after the block and its means or biases, a second row or a second octet need those.
  static constexpr int kVectors = POST && AFF && (GATE == kFullGate || GATE == kOneGate) ? 3
                                  : NV > 1 || (POST && AFF) || kTwoRows ? 2
                                                                             : 0;
  static constexpr int kFit =
      ring_stages(kPiecesRow, kBwdThreads,
                  kSmemPerSm - 4 * static_cast<int>(kTailBytes) - kVectors * NV * kBwdThreads * 32,
                  4);
  static constexpr int kRows = kTwoRows && kFit >= 4 ? 2 : 1;
  static constexpr int kStages = kFit / kRows * kRows;
  // Two octets a thread: twice the sums over tokens in registers, and two stages.
  static constexpr bool kPossible = NV == 1 || (!(POST && AFF) && kStages >= 2);
  // Sums over tokens that a thread has; the groups' are added where the ring was.
  static constexpr int kTokenSums =
      1 + AFF + POST + (POST && AFF) + (GATE == kChannelGate ? 1 : 0);
  static_assert(!kPossible || kStages * kPiecesRow * 16 >= kTokenSums * NV * 32, "they fit");
};

// AFF: a mean or a bias is wanted.
template <class TY, class TH, bool POST, bool AFF, int GATE, int NV>
__global__ void __launch_bounds__(kBwdThreads, 1)
    resnorm_bwd_kernel(const __grid_constant__ NormParams p) {
  __shared__ float slots[kMaxRowWarps][2][kMaxSums][kMaxRowWarps];
  __shared__ float cluster_slots[2][4][kMaxSums];
  __shared__ float ones[kMaxRowWarps];
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
  if (p.sums_follow) grid_launch_dependents();  // their CTAs take the SMs that this launch's leave
  using Shape = BwdShape<TY, TH, POST, AFF, GATE, NV>;
  // this thread's octets: of those of its CTA, and of the row
  const int jump = 32 * p.warps;
  const int mine = p.octets < p.H / 8 - rank * p.octets ? p.octets : p.H / 8 - rank * p.octets;
  int in_cta[NV], oct[NV];
  bool in[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    in_cta[j] = j * jump + sums.warp * 32 + lane;
    oct[j] = rank * p.octets + in_cta[j];
    in[j] = in_cta[j] < mine;
  }
  const bool pfp = p.params_fp32, layer = p.layer;
  constexpr bool kReadsY = POST || GATE != kNoGate;
  constexpr bool kBf16 = Elem<TH>::kBytes == 2;
  // a is the same in every row, so that it and the weight multiply the sums, not the rows
  constexpr bool kFixed = GATE == kNoGate || GATE == kChannelGate;

  const int64_t unit = static_cast<int64_t>(blockIdx.x / p.cluster) * p.groups + group;
  const int64_t units = static_cast<int64_t>(gridDim.x / p.cluster) * p.groups;
  const uint32_t step = blockDim.x * 16;
  const uint32_t ring = smem_addr(ring_raw);
  constexpr int R = Shape::kRows;
  constexpr int kStages = Shape::kStages;
  const uint32_t per_octet = step * (Shape::kPiecesRow / NV);
  const uint32_t tail = per_octet * NV, stage = tail + kTailBytes;
  const uint32_t end = kStages * stage;
  const uint32_t my_tail = smem_addr(ring_raw) + tail + warp * kRowBytes;
  const uint32_t at_h = kPieces<TY> * step, at_dh = at_h + kPieces<TH> * step;
  const uint32_t at_y = at_dh + kPieces<TH> * step, at_gate = at_y + kPieces<TY> * step;
  constexpr bool kOwn = Slot<TY>::kOwn && Slot<TH>::kOwn;
  int64_t ahead = unit;
  Walk<TY> dz_in(p.dz.p, p.dz.row, unit, oct[0]), y_in(p.y.p, p.y.row, unit, oct[0]);
  Walk<TH> h_in(p.h_out.p, p.h_out.row, unit, oct[0]);
  Walk<TH> dh_in(p.dh_out.p, p.dh_out.row, unit, oct[0]);
  Walk<TY> gate_in(p.gate.p, p.gate.row, unit, oct[0]);
  const bool token = GATE == kOneGate && p.gate_kind == FLCE_GATE_TOKEN;
  // address of a token's gate; its word, if all of that belongs to some token
  auto gate_of = [&](int64_t row) {
    return static_cast<const uint8_t*>(p.gate.p) + row * p.gate.row * Elem<TY>::kBytes;
  };
  auto fetch = [&](uint32_t s) {
    if (ahead < p.N) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const uint32_t at = ring + s + j * per_octet;
        const Slot<TY> slot_y(threadIdx.x, lane, in_cta[j], mine);
        const Slot<TH> slot_h(threadIdx.x, lane, in_cta[j], mine);
        const int y_on = j * jump * 8 * Elem<TY>::kBytes, h_on = j * jump * 8 * Elem<TH>::kBytes;
        // one branch for all copies where a lane makes all of its own or none
        if (kOwn && !in[j]) continue;
        if (p.pre) {
          slot_y.copy(at, dz_in.at + y_on, kOwn);
          slot_h.copy(at + at_h, h_in.at + h_on, kOwn);
        }
        if (p.dh_out.p) slot_h.copy(at + at_dh, dh_in.at + h_on, kOwn);
        if (kReadsY) slot_y.copy(at + at_y, y_in.at + y_on, kOwn);
        if (GATE == kFullGate) slot_y.copy(at + at_gate, gate_in.at + y_on, kOwn);
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
  // Single bf16 rows that are not read again ask for the next ones behind the exchange of their
  // sums, between their own loads and stores, when their own stage is free too: 65536 x 4096
  // 390 us, 415 with the copies first; with gates per element, sigmoids, 641 and 705; 30000 x 1000 55
  // either way.  (Pairs of rows 79 and 74 at 8192 x 4096, two octets a thread 67 and 58 at
  // 4096 x 8192; with an fp32 stream, or means on both sides, up to 4% more.)
  constexpr bool kAgain = R > 1 || NV > 1;
  constexpr bool kLate = !kAgain && Elem<TH>::kBytes == 2 && !(POST && AFF);
  constexpr int kAhead = kLate ? kStages : kStages - R;
  uint32_t s_in = 0, s_out = 0;
  for (; s_in < kAhead * stage; s_in += stage) fetch(s_in);
  if (s_in == end) s_in = 0;
  auto gate_of_channel = [&](int j) {  // act(gate), 1 without one
    if (GATE != kChannelGate) return same_oct(1.f);
    return gate_act_oct(p.act, param_octet<TY>(p.gate.p, pfp, oct[j], 1.f));
  };
  // w_post and b_post: times beta, and a where that is fixed
  constexpr bool kShared = Shape::kVectors > 0;
  const uint32_t plane = NV * jump * 16;
  const uint32_t vectors = smem_addr(ring_raw) + end + in_cta[0] * 16;
  Oct w_pre = zero_oct(), w_post = zero_oct();
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    Oct b_post = zero_oct();
    w_pre = w_post = zero_oct();
    if (in[j]) {
      w_pre = param_octet<TY>(p.w_pre, pfp, oct[j], 1.f);
      w_post = param_octet<TY>(POST ? p.w_post : nullptr, pfp, oct[j], 1.f);
      if (kFixed) scale_oct(w_post, gate_of_channel(j));
      scale_oct(w_post, p.beta);
      if (Shape::kVectors == 3) {
        b_post = param_octet<TY>(p.b_post, pfp, oct[j], 0.f);
        scale_oct(b_post, p.beta);
      }
    }
    if (kShared && group == 0) {
      const uint32_t to = vectors + j * jump * 16;
      put_shared(to, plane, w_pre);
      put_shared(to + 2 * plane, plane, w_post);
      if (Shape::kVectors == 3) put_shared(to + 4 * plane, plane, b_post);
    }
  }
  if (kShared) __syncthreads();
  auto vector = [&](int k, int j) {
    return shared_oct(vectors + 2 * k * plane + j * jump * 16, plane);
  };
  auto pre_weight = [&](int j) { return kShared ? vector(0, j) : w_pre; };
  auto post_weight = [&](int j) { return kShared ? vector(1, j) : w_post; };
  float scalar = 0.f;
  if (GATE == kOneGate && !token) scalar = gate_act(p.act, one_element<TY>(p.gate.p, pfp, 0));

  // Sums over tokens: dz xh, dz, and yh du, du without the factor beta and a fixed gate's.
  Oct s_pre[NV], s_bpre[NV], s_post[NV], s_bpost[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) s_pre[j] = s_bpre[j] = s_post[j] = s_bpost[j] = zero_oct();
  float s_one = 0.f;
  // Sum of w over a row, where w is the same in every row.
  constexpr bool kSumW = POST && AFF && GATE != kFullGate;
  float sum_w = 0.f;
  if (kSumW) {
    float t[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) t[0] += sum_oct(post_weight(j));
    sums.add(t);
    more.add(t);
    sum_w = t[0];
  }
  // The gradient of a gate of one value has sum b_post dt in it, which needs the sums of its
  // row: it is taken with the next row's.
  constexpr bool kCarry = kSumW && GATE == kOneGate;
  float carry = 0.f, wyd_before = 0.f, one_before = 0.f;
  auto put_one = [&](int64_t row, float wyd, float act) {
    if (!token)
      s_one += wyd;
    else if (in_cta[0] == 0 && rank == 0)
      store_element(TY{}, p.dgate.p, row * p.dgate.row, wyd * gate_slope(p.act, act));
  };
  Walk<TY> dy(p.dy.p, p.dy.row, unit, oct[0]), dgate(p.dgate.p, p.dgate.row, unit, oct[0]);
  Walk<TH> dh(p.dh.p, p.dh.row, unit, oct[0]);
  const GateSlope slope(p.act);
  for (int64_t row = unit; row < p.N; row += R * units) {
    auto fetch_rows = [&] {
#pragma unroll
      for (int q = 0; q < R; ++q) fetch(s_in + q * stage);
      s_in = s_in + R * stage == end ? 0 : s_in + R * stage;
    };
    if (!kLate) fetch_rows();
    auto there = [&](int q, int j) { return in[j] && (q == 0 || row + q * units < p.N); };
    copies_wait<kStages - R>();
    __syncwarp();  // lanes read what others copied

    Oct dz, xh, e, yh, a = zero_oct();
    float one = 0.f;  // act(gate) of gates with one value; `a` of those per element
    float mean_y = 0.f, r_y = 1.f, mean_h = 0.f, r_h = 0.f, rs_y[R] = {}, rs_h[R] = {};
    // dz, xh, dh' and yh of row q's octet j; a second time where two are in hand, which
    // takes fewer registers than keeping them
    const Slot<TY> slot_y(threadIdx.x, lane, 0, 0);
    const Slot<TH> slot_h(threadIdx.x, lane, 0, 0);
    auto read = [&](int q, int j, bool again) {
      const uint32_t at = ring + s_out + q * stage + j * per_octet;
      const uint32_t row_at = my_tail + s_out + q * stage;
      if (again) {
        if (R > 1) {  // of RMS norms
          r_y = rs_y[q];
          r_h = rs_h[q];
        }
      } else if (j == 0) {
        const uint4 t = ld_shared16(row_at);
        mean_y = AFF ? __uint_as_float(t.x) : 0.f;
        rs_y[q] = r_y = __uint_as_float(t.y);
        mean_h = AFF ? __uint_as_float(t.z) : 0.f;
        rs_h[q] = r_h =
            p.pre && (q == 0 || row + q * units < p.N) ? __uint_as_float(t.w) : 0.f;
        if (GATE == kOneGate) {
          one = scalar;
          if (token) {
            const uint32_t w = ld_shared4(row_at + 16);
            const bool upper = Elem<TY>::kBytes == 2 &&
                               (reinterpret_cast<uintptr_t>(gate_of(row + q * units)) & 2);
            one = gate_act(p.act, element_value<TY>(upper ? w >> 16 : w, false));
          }
        }
      }
      dz = xh = e = yh = a = zero_oct();
      if (there(q, j)) {
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
        if (GATE == kFullGate) a = gate_act_each<kBf16>(p.act, slot_y.read(at + at_gate));
      }
    };
    // Sums of a row: g xh, [g]; and with a post-norm or a gate of one value, with w for
    // beta [a] w_post: w yh e, w yh xh, [w yh], and for layer norms [w e, w, w xh].  Where
    // sum w is known, the row before's b_post dt takes its place.
    constexpr bool kSumsY = POST || GATE == kOneGate;
    constexpr int K = kSumsY ? (AFF ? 8 : 4) : (AFF ? 2 : 1);
    float s[R * K];
#pragma unroll
    for (int q = 0; q < R; ++q) {
      float2 v[K];
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] = pair(0.f);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        read(q, j, false);
        const Oct wp = pre_weight(j), wq = post_weight(j);
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
              if (!kSumW) v[5] = plus2(v[5], w);
              v[6] = mad2(w, xh.p[i], v[6]);
            }
          }
        }
      }
#pragma unroll
      for (int k = 0; k < K; ++k) s[q * K + k] = v[k].x + v[k].y;
    }
    if (kCarry) s[5] = carry;
    // (the exchanges also see to it that all lanes have read what later copies overwrite)
    if (p.pre || kSumsY) {
      sums.add(s);
      more.add(s);
    } else {
      __syncwarp();
    }
    if (kCarry && row != unit) put_one(row - units, wyd_before + s[5], one_before);

    if (kLate) fetch_rows();
#pragma unroll
    for (int q = 0; q < R; ++q) {
      float c1 = 0.f, c2 = 0.f, m1 = 0.f, m2 = 0.f, wyd = 0.f;
      carry = kCarry ? 0.f : carry;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (kAgain) {
          read(q, j, true);
          if (!kOwn && q == R - 1 && j == NV - 1) __syncwarp();  // as above
        }
        if (j == 0) {
          m2 = r_h * s[q * K] * p.inv_h;
          m1 = AFF && layer ? r_h * s[q * K + K - 1] * p.inv_h : 0.f;
          // sum w yh dt: with a gate of one value its gradient, and dy's second mean
          if (kSumsY) wyd = s[q * K + 1] - m2 * s[q * K + 2] - (AFF ? m1 * s[q * K + 3] : 0.f);
          if (POST) {
            c2 = r_y * p.inv_h * wyd;
            if (AFF && layer)
              c1 = r_y * p.inv_h * (s[q * K + 4] - m2 * s[q * K + 6] -
                                      m1 * (kSumW ? sum_w : s[q * K + 5]));
          }
          if (GATE == kOneGate) {
            c1 *= one;
            c2 *= one;
          }
        }
        const Oct wp = kAgain ? pre_weight(j) : zero_oct(), wq = post_weight(j);
        const Oct bq = Shape::kVectors == 3 ? vector(2, j) : zero_oct();
        Oct dg = zero_oct();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (kAgain) e.p[i] = mad2(pair(r_h), mul2(dz.p[i], wp.p[i]), e.p[i]);
          float2 dt = mad2(pair(-m2), xh.p[i], e.p[i]);
          if (AFF) dt = plus2(dt, pair(-m1));
          s_pre[j].p[i] = mad2(dz.p[i], xh.p[i], s_pre[j].p[i]);
          if (AFF) s_bpre[j].p[i] = plus2(s_bpre[j].p[i], dz.p[i]);
          // du over beta, or beta a where that is fixed
          float2 du = dt;
          if (GATE == kOneGate) du = mul2(pair(one), dt);
          if (GATE == kFullGate) {
            du = mul2(a.p[i], dt);
            // beta u: w_post is times beta, and beta itself without a post-norm
            const float2 u = Shape::kVectors == 3 ? mad2(yh.p[i], wq.p[i], bq.p[i])
                                                  : mul2(yh.p[i], wq.p[i]);
            dg.p[i] = mul2(mul2(slope(a.p[i]), u), dt);
          }
          if (POST || GATE == kChannelGate) s_post[j].p[i] = mad2(yh.p[i], du, s_post[j].p[i]);
          if (POST && AFF) s_bpost[j].p[i] = plus2(s_bpost[j].p[i], du);
          float2 gy = mul2(wq.p[i], du);
          if (POST) {
            gy = mad2(pair(-c2), yh.p[i], mul2(pair(r_y), gy));
            if (AFF) gy = plus2(gy, pair(-c1));
          }
          e.p[i] = gy;                        // dy
          if (kCarry) a.p[i] = mul2(bq.p[i], dt);
          xh.p[i] = mul2(pair(p.alpha), dt);  // dh
        }
        if (kCarry) carry += sum_oct(a);
        const int y_on = j * jump * 8 * Elem<TY>::kBytes, h_on = j * jump * 8 * Elem<TH>::kBytes;
        if (there(q, j)) {
          dy.put(to_octet(TY{}, e), p.wide, y_on);
          if (p.dh.p) dh.put(to_octet(TH{}, xh), p.wide, h_on);
          if (GATE == kFullGate) dgate.put(to_octet(TY{}, dg), p.wide, y_on);
        }
      }
      dy.at += p.dy.step;
      dh.at += p.dh.step;
      if (GATE == kFullGate) dgate.at += p.dgate.step;
      if (kCarry) {
        wyd_before = wyd;
        one_before = one;
      } else if (GATE == kOneGate) {
        put_one(row + q * units, wyd, one);
      }
    }
    s_out = s_out + R * stage == end ? 0 : s_out + R * stage;
  }

  if (kCarry && unit < p.N) {
    float t[1] = {carry};
    sums.add(t);
    more.add(t);
    // of the last row, which is the units before the first that there is not
    put_one(unit + (p.N - 1 - unit) / units * units, wyd_before + t[0], one_before);
  }

  // The groups' sums over tokens, then the CTA's, in order of the groups.
  const int64_t part_row = blockIdx.x / p.cluster;
  const bool alone = p.groups == 1;
  const uint32_t planes = ring + in_cta[0] * 16;
  auto place = [&](int k, int g, int j) {
    return planes + 2 * plane * (k * p.groups + g) + j * jump * 16;
  };
  if (!alone) {
    copies_wait<0>();
    __syncthreads();  // all have left the ring
  }
  constexpr int kBpre = 1, kGate = 1 + AFF, kPost = kGate + (GATE == kChannelGate ? 1 : 0);
  float* to[5] = {p.part[0]};  // by plane
  if (AFF) to[kBpre] = p.part[1];
  if (GATE == kChannelGate) to[kGate] = p.part[4];
  if (POST) to[kPost] = p.part[2];
  if (POST && AFF) to[kPost + 1] = p.part[3];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    auto put = [&](int k, const Oct& o) {
      if (!to[k] || !in[j]) return;
      if (alone) store_octet<float>(to[k] + part_row * p.H, oct[j], o);
      else put_shared(place(k, group, j), plane, o);
    };
    put(0, s_pre[j]);
    if (AFF) put(kBpre, s_bpre[j]);
    if (kFixed && kReadsY && in[j]) {
      const Oct a = gate_of_channel(j);
      if (GATE == kChannelGate) {
        // dgate = slope (w_post sum yh dt + b_post sum dt)
        Oct f = param_octet<TY>(POST ? p.w_post : nullptr, pfp, oct[j], 1.f);
        scale_oct(f, s_post[j]);
        if (POST && AFF) {
          const Oct b = param_octet<TY>(p.b_post, pfp, oct[j], 0.f);
#pragma unroll
          for (int i = 0; i < 4; ++i) f.p[i] = mad2(b.p[i], s_bpost[j].p[i], f.p[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          f.p[i] = mul2(f.p[i], make_float2(p.beta * gate_slope(p.act, a.p[i].x),
                                            p.beta * gate_slope(p.act, a.p[i].y)));
        put(kGate, f);
      }
      scale_oct(s_post[j], a);
      scale_oct(s_bpost[j], a);
    }
    scale_oct(s_post[j], p.beta);
    scale_oct(s_bpost[j], p.beta);
    if (POST) put(kPost, s_post[j]);
    if (POST && AFF) put(kPost + 1, s_bpost[j]);
  }
  if (GATE == kOneGate && in_cta[0] == 0) ones[group] = s_one * gate_slope(p.act, scalar);
  if (!alone || GATE == kOneGate) __syncthreads();
  if (!alone) {
#pragma unroll
    for (int k = 0; k < Shape::kTokenSums; ++k) {
      if (k % p.groups != group || !to[k]) continue;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (!in[j]) continue;
        Oct o = shared_oct(place(k, 0, j), plane);
        for (int g = 1; g < p.groups; ++g) {
          const Oct t = shared_oct(place(k, g, j), plane);
#pragma unroll
          for (int i = 0; i < 4; ++i) o.p[i] = plus2(o.p[i], t.p[i]);
        }
        store_octet<float>(to[k] + part_row * p.H, oct[j], o);
      }
    }
  }
  if (GATE == kOneGate && p.part[4] && threadIdx.x == 0 && rank == 0) {
    float v = ones[0];
    for (int g = 1; g < p.groups; ++g) v += ones[g];
    p.part[4][part_row] = v;
  }
  if (p.cluster > 1) cluster_sync();  // no CTA leaves while another writes to its slots
}

// With parts == 0, sets p.fit, the clusters that run at once: of four CTAs fewer than the SMs
// would make, as a cluster stays within one of the device's processor clusters.
template <class TY, class TH, bool POST, bool AFF, int GATE, int NV>
cudaError_t launch_bwd_nv(NormParams& p, int64_t parts, cudaStream_t s) {
  using Shape = BwdShape<TY, TH, POST, AFF, GATE, NV>;
  static SmemLimit limit;
  const int threads = 32 * p.warps * p.groups;
  const int vectors = Shape::kVectors * NV * 32 * p.warps * 32;
  const int ring = (threads * 16 * Shape::kPiecesRow + static_cast<int>(kTailBytes)) * Shape::kStages;
  const auto kernel = resnorm_bwd_kernel<TY, TH, POST, AFF, GATE, NV>;
  cudaError_t e = limit.raise(kernel, kSmemPerSm);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(static_cast<unsigned>((parts ? parts : 1) * p.cluster));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(ring + vectors);
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(p.cluster);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (parts == 0) {
    p.fit = p.sms;
    if (p.cluster == 1) return cudaSuccess;
    // of a CTA at its largest, so that the order of the sums does not go by earlier calls
    cfg.blockDim = dim3(kBwdThreads);
    cfg.dynamicSmemBytes = kSmemPerSm;
    static std::atomic<int> known[64][2];  // by device and size
    int dev = 0, n = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    std::atomic<int>& at = known[dev & 63][p.cluster == 4];
    n = at.load(std::memory_order_relaxed);
    if (n == 0) {
      if ((e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg)) != cudaSuccess) return e;
      if (n < 1) n = 1;
      at.store(n, std::memory_order_relaxed);
    }
    p.fit = n;
    return cudaSuccess;
  }
  set_steps(p, parts * p.groups, Elem<TY>::kBytes, Elem<TH>::kBytes);
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// Warps of 16 that are busy with rows of `octets` octets, NV of them a thread.
inline int busy_warps(int octets, int nv) {
  const int warps = (octets + 32 * nv - 1) / (32 * nv);
  return kMaxRowWarps / warps * warps;
}

// The launch's shape: two octets a thread where that spares a cluster (4096 x 8192: 74 us, 104
// with a cluster of two) or keeps half as many warps again busy (16000 x 2056: 9 of 16 with
// one, 118 us; 15 with two, 92).
inline void plan_bwd(NormParams& p, bool two) {
  const int octets = p.H / 8;
  const int nv = two && (octets > 32 * kMaxRowWarps ||
                         2 * busy_warps(octets, 2) >= 3 * busy_warps(octets, 1))
                     ? 2
                     : 1;
  const int most = 32 * kMaxRowWarps * nv;
  p.nv = nv;
  p.cluster = octets <= most ? 1 : octets <= 2 * most ? 2 : 4;
  p.octets = (octets + p.cluster - 1) / p.cluster;
  p.warps = (p.octets + 32 * nv - 1) / (32 * nv);
  p.groups = kMaxRowWarps / p.warps;
}

// parts == 0: sets the launch's shape only.
template <class TY, class TH, bool POST, bool AFF, int GATE>
cudaError_t launch_bwd(NormParams& p, int64_t parts, cudaStream_t s) {
  constexpr bool kTwo = BwdShape<TY, TH, POST, AFF, GATE, 2>::kPossible;
  if (parts == 0) plan_bwd(p, kTwo);
  if constexpr (kTwo)
    if (p.nv == 2) return launch_bwd_nv<TY, TH, POST, AFF, GATE, 2>(p, parts, s);
  return launch_bwd_nv<TY, TH, POST, AFF, GATE, 1>(p, parts, s);
}

template <class TY, class TH, bool POST, bool AFF>
cudaError_t launch_bwd_gate(NormParams& p, int64_t parts, cudaStream_t s) {
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
cudaError_t launch_bwd_types(NormParams& p, int64_t parts, cudaStream_t s) {
  if (p.post)
    return p.biased ? launch_bwd_gate<TY, TH, true, true>(p, parts, s)
                    : launch_bwd_gate<TY, TH, true, false>(p, parts, s);
  return p.biased ? launch_bwd_gate<TY, TH, false, true>(p, parts, s)
                  : launch_bwd_gate<TY, TH, false, false>(p, parts, s);
}

}  // namespace flce
