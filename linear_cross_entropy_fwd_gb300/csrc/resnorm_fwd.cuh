// resnorm_fwd.cuh -- the residual join's forward pass (resnorm.h has the formulas); one
// translation unit per pair of types includes it.
//
// Bound by memory: a token's y and h are read once and h', z written once.  `warps` warps
// hold a row in registers, NV octets a thread, and a CTA has several rows at a time when
// they are short; the next rows are on their way into shared memory meanwhile (Ring in
// rows.cuh).  A mean and a variance are two sums one after the other, so that nothing
// cancels; RMS norms need one.  A row may hold anything finite.
//
// 8192 x 4096 in bf16: 46 us with an RMS norm before the next block (5.8 TB/s), 48 with one on
// both sides (32768 x 4096: 161 and 165, 6.6 TB/s), 51 with a layer norm, 68 with two and their
// biases, whose four exchanges per pair of rows are then the bound; fp32 throughout 95 us (5.7
// TB/s).  One token takes 4.5 us, a launch's latency.  With a checkpoint of z the first two take 51
// and 57 us, where saving it afterwards takes 15 and 19 more.
#pragma once
#include "host_util.h"
#include "resnorm.h"

namespace flce {

constexpr int kFwdThreads = 512;

// Sums of (x - mean)^2 over R rows; places behind their end hold 0 and stay out of it.
template <int R, int NV, bool LAYER>
__device__ __forceinline__ void squares(const Oct (&x)[R][NV], const bool (&in)[NV],
                                        const float (&mean)[R], RowSums& sums, float (&v)[R]) {
#pragma unroll
  for (int q = 0; q < R; ++q) {
    float2 s = pair(0.f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (LAYER && !in[j]) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 d = LAYER ? plus2(x[q][j].p[i], pair(-mean[q])) : x[q][j].p[i];
        s = mad2(d, d, s);
      }
    }
    v[q] = s.x + s.y;
  }
  sums.add(v);
}

// x -> x - mean in place over R rows, with mean and r for the statistics; f makes n(x) of it.
template <int R, int NV, bool LAYER>
__device__ __forceinline__ void normalise(Oct (&x)[R][NV], const bool (&in)[NV], float eps,
                                          float inv_h, RowSums& sums, float (&mean)[R],
                                          float (&r)[R], float (&f)[R]) {
  float m[R], v[R], scale[R];
#pragma unroll
  for (int q = 0; q < R; ++q) scale[q] = 1.f;
  for (int again = 0;; again = 1) {
#pragma unroll
    for (int q = 0; q < R; ++q) m[q] = 0.f;
    if (LAYER) {
#pragma unroll
      for (int q = 0; q < R; ++q)
#pragma unroll
        for (int j = 0; j < NV; ++j) m[q] += sum_oct(x[q][j]);
      sums.add(m);
#pragma unroll
      for (int q = 0; q < R; ++q) m[q] *= inv_h;
    }
    squares<R, NV, LAYER>(x, in, m, sums, v);
    bool fine = true;
#pragma unroll
    for (int q = 0; q < R; ++q) {
      v[q] = fmaf(v[q], inv_h, eps * scale[q] * scale[q]);
      fine = fine && v[q] < 1e38f && v[q] >= 1e-30f;
    }
    if (__builtin_expect(fine || again, 1)) break;
    // Squares beyond fp32's range: the row times a power of two, whose squares are not.  (With
    // an eps above 1e-30, squares that vanish beside it need nothing.)
#pragma unroll
    for (int q = 0; q < R; ++q) {
      float top = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          top = fmaxf(top, fmaxf(fabsf(x[q][j].p[i].x), fabsf(x[q][j].p[i].y)));
      top = sums.max(top);
      if (v[q] < 1e38f && v[q] >= 1e-30f) continue;  // its bits do not go by its neighbour
      const int k = min(max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -100), 126);
      scale[q] = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
#pragma unroll
      for (int j = 0; j < NV; ++j) scale_oct(x[q][j], scale[q]);
    }
  }
#pragma unroll
  for (int q = 0; q < R; ++q) {
    f[q] = rsqrtf(v[q]);
    if (LAYER) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[q][j].p[i] = plus2(x[q][j].p[i], pair(-m[q]));
    }
    mean[q] = LAYER ? m[q] / scale[q] : 0.f;
    r[q] = f[q] * scale[q];
  }
}

// Biases wait in shared memory behind the ring: read again from where they are, they took
// a third of the time (8192 x 4096, layer norms on both sides: 97 us, 68 now).
template <int NV, bool FULL>
constexpr bool kBiasShared = NV <= 2 && !FULL;
// Stages of the ring: a row's y, h and, FULL, a gate per element.
template <class TY, class TH, int NV, bool FULL>
constexpr int kFwdStages = ring_stages(
    NV * (kPieces<TY> * (FULL ? 2 : 1) + kPieces<TH>), kFwdThreads,
    kSmemPerSm - (kBiasShared<NV, FULL> ? 2 * NV * kFwdThreads * 32 : NV == 4 && !FULL ? kMaxH * 4 : 0),
    6);
// Rows that a group takes at a time: two share the instructions around them and the
// exchanges of their sums (8192 x 4096 in bf16 with both norms: 55 us with one, 46).
template <class TY, class TH, int NV, bool FULL>
constexpr int kFwdRows = NV <= 2 && kFwdStages<TY, TH, NV, FULL> >= 4 ? 2 : 1;

// Without a norm after the block h' follows its loads at once, and many rows in bf16 take less
// time when the next ones are asked for behind it (LATE), not before: 32768 x 4096 161 us
// against 187, 12288 x 4096 65 against 71, with a gate per element 81 either way, 6144 x 4096 36
// against 35.  (With that norm, which keeps loads and stores apart, 182 against 165 at 32768;
// with layer norms or an fp32 stream no gain.)
template <class TY, class TH, int NV, bool LAYER, bool FULL>
constexpr bool kMayBeLate = NV == 2 && !LAYER && Elem<TH>::kBytes == 2 &&
                            kFwdRows<TY, TH, NV, FULL> == 2;
constexpr int kLateRows = 40;  // of a group of warps, at least

// LATE: without a norm after the block.
template <class TY, class TH, int NV, bool LAYER, bool FULL, bool LATE>
__global__ void __launch_bounds__(kFwdThreads, 1)
    resnorm_fwd_kernel(const __grid_constant__ NormParams p) {
  __shared__ float slots[kMaxRowWarps][2][kMaxSums][kMaxRowWarps];
  extern __shared__ __align__(16) uint8_t ring_raw[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int group = warp / p.warps;
  RowSums sums{slots[group], p.warps, warp - group * p.warps, group, 0};
  const int octets = p.H / 8;
  int oct[NV];
  bool in[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    oct[j] = (j * p.warps + sums.warp) * 32 + lane;
    in[j] = oct[j] < octets;
  }
  const int jump = p.warps * 32;  // octets from one of a thread's to the next
  const bool pfp = p.params_fp32;
  constexpr bool kBf16 = Elem<TH>::kBytes == 2;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * p.groups + group;
  const int64_t rows = static_cast<int64_t>(gridDim.x) * p.groups;

  // The ring: of each of a thread's octets y, then h, then a gate per element.
  const uint32_t step = blockDim.x * 16;
  const uint32_t ring = smem_addr(ring_raw);
  constexpr int kPer = kPieces<TY> + kPieces<TH> + (FULL ? kPieces<TY> : 0);
  const uint32_t at_h = kPieces<TY> * step, at_gate = at_h + kPieces<TH> * step;
  constexpr int R = kFwdRows<TY, TH, NV, FULL>;
  constexpr int kStages = kFwdStages<TY, TH, NV, FULL> / R * R;
  static_assert(kStages >= 1, "a stage of the longest row");
  const uint32_t stage = step * NV * kPer, end = kStages * stage;
  int64_t ahead = first;
  Walk<TY> y(p.y.p, p.y.row, first, oct[0]), gate(p.gate.p, p.gate.row, first, oct[0]);
  Walk<TH> h(p.h.p, p.h.row, first, oct[0]);
  auto fetch = [&](uint32_t s) {
    if (ahead < p.N) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const uint32_t to = ring + s + j * kPer * step;
        const Slot<TY> slot_y(threadIdx.x, lane, oct[j], octets);
        const Slot<TH> slot_h(threadIdx.x, lane, oct[j], octets);
        constexpr bool kOwn = Slot<TY>::kOwn && Slot<TH>::kOwn;
        if (kOwn && !in[j]) continue;
        slot_y.copy(to, y.at + j * jump * 8 * Elem<TY>::kBytes, kOwn);
        if (p.h.p) slot_h.copy(to + at_h, h.at + j * jump * 8 * Elem<TH>::kBytes, kOwn);
        if (FULL) slot_y.copy(to + at_gate, gate.at + j * jump * 8 * Elem<TY>::kBytes, kOwn);
      }
      ahead += rows;
      y.at += p.y.step;
      h.at += p.h.step;
      if (FULL) gate.at += p.gate.step;
    }
    copies_commit();
  };
  uint32_t s_in = 0, s_out = 0;
  for (; s_in < end - R * stage; s_in += stage) fetch(s_in);

  for (int i = threadIdx.x; i < kMaxRowWarps * 2 * kMaxSums * kMaxRowWarps; i += blockDim.x)
    (&slots[0][0][0][0])[i] = 0.f;
  // What multiplies n(y) whatever the row: the weight, beta and a gate per channel; and what
  // is added, likewise (0 without a bias).  A thread keeps its octets' factors, and the other
  // norm's weights; of the longest rows they wait in shared memory behind the ring or, where
  // gates per element need that room, are read again.
  auto factor = [&](const void* w, float missing, int o) {
    Oct f = param_octet<TY>(w, pfp, o, missing);
    if (!FULL && p.gate_kind == FLCE_GATE_CHANNEL)
      scale_oct(f, gate_act_oct(p.act, param_octet<TY>(p.gate.p, pfp, o, 1.f)));
    scale_oct(f, p.beta);
    return f;
  };
  constexpr bool kKeep = NV <= 2, kBias = kBiasShared<NV, FULL>;
  const uint32_t factors = smem_addr(ring_raw) + end;
  const uint32_t plane = NV * jump * 16;
  const uint32_t biases = factors + oct[0] * 16;  // two planes each: b_post, b_pre
  Oct c[kKeep ? NV : 1], w_pre[kKeep ? NV : 1];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (kKeep) {
      c[j] = in[j] ? factor(p.w_post, 1.f, oct[j]) : zero_oct();
      w_pre[j] = in[j] ? param_octet<TY>(p.w_pre, pfp, oct[j], 1.f) : zero_oct();
    } else if (!FULL && in[j]) {
      store_octet<float>(ring_raw + end, oct[j], factor(p.w_post, 1.f, oct[j]));  // its own
    }
    if (kBias && group == 0 && in[j]) {
      if (p.b_post) put_shared(biases + j * jump * 16, plane, factor(p.b_post, 0.f, oct[j]));
      if (p.b_pre)
        put_shared(biases + 2 * plane + j * jump * 16, plane,
                   param_octet<TY>(p.b_pre, pfp, oct[j], 0.f));
    }
  }
  const bool token = p.gate_kind == FLCE_GATE_TOKEN;
  const bool one_gate = token || p.gate_kind == FLCE_GATE_SCALAR;
  // a gate with one value: its bits, a token's an iteration ahead (of the last row again
  // behind it, as a branch would wait for what it loads)
  uint32_t one[R];
#pragma unroll
  for (int q = 0; q < R; ++q) one[q] = 0;
  auto read_gates = [&](int64_t row) {
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const int64_t at = row + q * rows < p.N ? row + q * rows : p.N - 1;
      one[q] = element_bits<TY>(p.gate.p, false, at * p.gate.row);
    }
  };
  if (token) read_gates(first);
  float scalar = 0.f;
  if (one_gate && !token) scalar = one_element<TY>(p.gate.p, pfp, 0);
  Walk<TH> h_out(p.h_out.p, p.h_out.row, first, oct[0]);
  Walk<TY> z(p.z.p, p.z.row, first, oct[0]);
  __syncthreads();

  auto fetch_rows = [&] {
#pragma unroll
    for (int q = 0; q < R; ++q) fetch(s_in + q * stage);
    s_in = s_in + R * stage == end ? 0 : s_in + R * stage;
  };
  static_assert(!LATE || kStages >= 2 * R, "rows in hand and rows on their way");
  const bool post = !LATE && p.post;
  for (int64_t row = first; row < p.N; row += R * rows) {
    if (!LATE) fetch_rows();
    bool there[R];
    Oct x[R][NV];
    float gate1[R], mean_y[R], r_y[R], mean_h[R], r_h[R], f[R];
#pragma unroll
    for (int q = 0; q < R; ++q) {
      there[q] = q == 0 || row + q * rows < p.N;
      gate1[q] = token ? element_value<TY>(one[q], false) : scalar;
      mean_y[q] = r_y[q] = mean_h[q] = r_h[q] = 0.f;
    }
    if (token) read_gates(row + R * rows);
    copies_wait<kStages - R - (LATE ? R : 0)>();
    __syncwarp();  // lanes read what others copied
    const Slot<TY> slot_y(threadIdx.x, lane, 0, 0);
    const Slot<TH> slot_h(threadIdx.x, lane, 0, 0);
    const uint32_t at = ring + s_out;
    s_out = s_out + R * stage == end ? 0 : s_out + R * stage;
#pragma unroll
    for (int q = 0; q < R; ++q)
#pragma unroll
      for (int j = 0; j < NV; ++j)
        x[q][j] = in[j] && there[q] ? slot_y.read(at + q * stage + j * kPer * step) : zero_oct();
    if (post) normalise<R, NV, LAYER>(x, in, p.eps, p.inv_h, sums, mean_y, r_y, f);
#pragma unroll
    for (int q = 0; q < R; ++q)
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        Oct& v = x[q][j];
        if (!in[j] || !there[q]) {
          v = zero_oct();
          continue;
        }
        const uint32_t mine = at + q * stage + j * kPer * step;
        if (post) scale_oct(v, f[q]);
        scale_oct(v, kKeep  ? c[kKeep ? j : 0]
                     : FULL ? factor(p.w_post, 1.f, oct[j])
                            : shared_oct(factors + oct[j] * 32, 16));
        if (p.b_post)
          add_oct(v, kBias ? shared_oct(biases + j * jump * 16, plane)
                           : factor(p.b_post, 0.f, oct[j]));
        if (FULL)
          scale_oct(v, gate_act_each<kBf16>(p.act, slot_y.read(mine + at_gate)));
        if (one_gate) scale_oct(v, gate_act(p.act, gate1[q]));
        if (p.h.p) {
          const Oct t = slot_h.read(mine + at_h);
#pragma unroll
          for (int i = 0; i < 4; ++i) v.p[i] = mad2(pair(p.alpha), t.p[i], v.p[i]);
        }
        // the stream is what is stored of it; see flce_resnorm
        const auto o = to_octet(TH{}, v);
        if (p.h_out.p)
          h_out.put(o, p.wide, q * p.h_out.step + j * jump * 8 * Elem<TH>::kBytes);
        v = from_octet(o);
      }
    if (LATE) fetch_rows();
    // all lanes have read what later copies overwrite: here, or by the exchanges of sums
    if (!p.pre) __syncwarp();
    if (p.pre) {
      normalise<R, NV, LAYER>(x, in, p.eps, p.inv_h, sums, mean_h, r_h, f);
#pragma unroll
      for (int q = 0; q < R; ++q)
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          Oct& v = x[q][j];
          if (in[j]) {
            scale_oct(v, f[q]);
            scale_oct(v, kKeep ? w_pre[kKeep ? j : 0]
                               : param_octet<TY>(p.w_pre, pfp, oct[j], 1.f));
            if (p.b_pre)
              add_oct(v, kBias ? shared_oct(biases + 2 * plane + j * jump * 16, plane)
                               : param_octet<TY>(p.b_pre, pfp, oct[j], 0.f));
          } else {
            v = zero_oct();
          }
          if (!there[q]) continue;
          const auto o = to_octet(TY{}, v);
          if (in[j])
            z.put(o, p.wide, q * p.z.step + j * jump * 8 * Elem<TY>::kBytes);
          if (p.ckpt.codes) {
            const int64_t at_row = row + q * rows;
            ckpt_store_octet(p.ckpt, p.ckpt.codes + at_row * p.ckpt.pitch + oct[j] * 8,
                             p.ckpt.scales + at_row * p.ckpt.spitch, oct[j], o);
          }
        }
    }
    h_out.at += R * p.h_out.step;
    z.at += R * p.z.step;
    if (p.stats && lane == 0 && sums.warp == 0) {
#pragma unroll
      for (int q = 0; q < R; ++q) {
        if (!there[q]) continue;
        float* s = p.stats + row + q * rows;
        s[0] = mean_y[q];
        s[p.N] = r_y[q];
        s[2 * p.N] = mean_h[q];
        s[3 * p.N] = r_h[q];
      }
    }
  }
}

template <class TY, class TH, int NV, bool LAYER, bool FULL, bool LATE = false>
cudaError_t launch(NormParams p, int sms, cudaStream_t s) {
  static SmemLimit limit;
  const int octets = p.H / 8;
  p.warps = (octets + 32 * NV - 1) / (32 * NV);
  p.groups = kFwdThreads / 32 / p.warps;
  const int threads = 32 * p.warps * p.groups;
  constexpr int kStages =
      kFwdStages<TY, TH, NV, FULL> / kFwdRows<TY, TH, NV, FULL> * kFwdRows<TY, TH, NV, FULL>;
  const int stage = threads * 16 * NV * (kPieces<TY> * (FULL ? 2 : 1) + kPieces<TH>);
  const int factors = kBiasShared<NV, FULL> ? (p.b_post || p.b_pre ? 4 * NV * 32 * p.warps * 16 : 0)
                      : NV == 4 && !FULL    ? p.H * 4
                                            : 0;
  const int64_t want = (p.N + p.groups - 1) / p.groups;
  const int64_t grid = want < sms ? want : sms;
  if constexpr (!LATE && kMayBeLate<TY, TH, NV, LAYER, FULL>)
    if (!p.post && p.N >= kLateRows * grid * p.groups)
      return launch<TY, TH, NV, LAYER, FULL, true>(p, sms, s);
  const auto kernel = resnorm_fwd_kernel<TY, TH, NV, LAYER, FULL, LATE>;
  const cudaError_t e = limit.raise(kernel, kSmemPerSm);
  if (e != cudaSuccess) return e;
  set_steps(p, grid * p.groups, Elem<TY>::kBytes, Elem<TH>::kBytes);
  kernel<<<static_cast<unsigned>(grid), threads,
           static_cast<size_t>(kStages) * stage + factors, s>>>(p);
  return cudaGetLastError();
}

template <class TY, class TH, int NV>
cudaError_t launch_nv(const NormParams& p, int sms, cudaStream_t s) {
  if (p.gate_kind == FLCE_GATE_FULL)
    return p.layer ? launch<TY, TH, NV, true, true>(p, sms, s)
                   : launch<TY, TH, NV, false, true>(p, sms, s);
  return p.layer ? launch<TY, TH, NV, true, false>(p, sms, s)
                 : launch<TY, TH, NV, false, false>(p, sms, s);
}

template <class TY, class TH>
cudaError_t launch_fwd_types(const NormParams& p, int sms, cudaStream_t s) {
  if (p.H <= 256) return launch_nv<TY, TH, 1>(p, sms, s);
  return p.H <= 8192 ? launch_nv<TY, TH, 2>(p, sms, s) : launch_nv<TY, TH, 4>(p, sms, s);
}

}  // namespace flce
