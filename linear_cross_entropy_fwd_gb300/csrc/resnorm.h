// resnorm.h -- what the residual join's kernels and their host side share (internal).
//
// For a token, with n(x) = (x - mean) r, r = 1 / sqrt(mean((x - mean)^2) + eps) and mean = 0
// for the RMS norm:
//   yh = n(y), u = yh w_post + b_post   (without a post-norm: yh = u = y)
//   h' = alpha h + beta a u, a = act(gate), rounded to the stream's type
//   xh = n(h'), z = xh w_pre + b_pre
// and for the gradients, with g = dz w_pre:
//   dt = dh' + r (g - [layer] mean(g) - xh mean(g xh)),  dh = alpha dt
//   du = beta a dt,  dgate = beta act'(gate) u dt
//   dy = r_y (gy - [layer] mean(gy) - yh mean(gy yh)), gy = du w_post   (else dy = du)
//   dw_pre = sum dz xh, db_pre = sum dz, dw_post = sum du yh, db_post = sum du over tokens.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/flce.h"
#include "ckpt.cuh"

namespace flce {

struct RowTensor {
  void* p;
  int64_t row;   // stride in elements
  int64_t step;  // bytes from a row to the next one of the same warps
};

struct NormParams {
  int64_t N;
  int32_t H;
  int32_t layer, post, pre, params_fp32;
  int32_t gate_kind, act;
  int32_t biased;      // backward: a mean or a bias is wanted
  int32_t wide;        // fp32 rows that are written are 32-byte aligned
  float alpha, beta, eps, inv_h;
  RowTensor y, h, gate, h_out, z, dz, dh_out, dy, dh, dgate;
  const void *w_post, *b_post, *w_pre, *b_pre;
  float* stats;        // [4][N]
  Ckpt ckpt;           // forward; codes null: none
  // launch shape
  int32_t warps;       // that share a row (of each CTA of a cluster)
  int32_t groups;      // rows of a CTA at a time
  // backward
  int32_t cluster;     // CTAs that share a row
  int32_t octets;      // of a row in each CTA of a cluster
  int32_t nv;          // octets of a thread
  int32_t sms, fit;    // of the device; CTAs or clusters that run at once
  int32_t sums_follow; // the next launch is launch_resnorm_sums
  float* part[5];      // sums over tokens of dw_pre, db_pre, dw_post, db_post, dgate:
                       // [parts][H], or [parts] for a scalar gate; null: not wanted
};

// The steps of a launch whose warps take every `rows`-th row.
inline void set_steps(NormParams& p, int64_t rows, int y_bytes, int h_bytes) {
  for (RowTensor* t : {&p.y, &p.gate, &p.z, &p.dz, &p.dy, &p.dgate}) t->step = rows * t->row * y_bytes;
  for (RowTensor* t : {&p.h, &p.h_out, &p.dh_out, &p.dh}) t->step = rows * t->row * h_bytes;
}

constexpr int kMaxH = 16384;
constexpr int kSmemPerSm = 208 << 10;  // for rings, beside the slots of the sums

cudaError_t launch_resnorm_fwd_bf16(const NormParams& p, int sms, cudaStream_t s);
cudaError_t launch_resnorm_fwd_mixed(const NormParams& p, int sms, cudaStream_t s);
cudaError_t launch_resnorm_fwd_fp32(const NormParams& p, int sms, cudaStream_t s);

// With parts == 0, the launch's shape is set and nothing is run; else `parts` is the number of
// rows of each of part[]: the grid's CTAs or clusters.
cudaError_t launch_resnorm_bwd_bf16(NormParams& p, int64_t parts, cudaStream_t s);
cudaError_t launch_resnorm_bwd_mixed(NormParams& p, int64_t parts, cudaStream_t s);
cudaError_t launch_resnorm_bwd_fp32(NormParams& p, int64_t parts, cudaStream_t s);

// out[k][col] = sum over `parts` rows of part[k], fp32, in a fixed order.
struct NormSums {
  const float* part[5];
  float* out[5];
  int32_t width[5];  // columns; 0: not wanted
  int64_t parts;
};
cudaError_t launch_resnorm_sums(const NormSums& p, cudaStream_t s);

// act(g), and its derivative by act(g).  The sigmoid is e or 1 over 1 + e, e = exp(-|g|), so that
// nothing overflows and numbers down to fp32's smallest are kept: off by 3.5 units in the last
// place at most (the exponential 1, the sum half of one, the quotient by a number in 1 .. 2 two).
// tanhf is within 2.
__device__ __forceinline__ float sigmoid_of(float g, float e) {
  return __fdividef(g >= 0.f ? 1.f : e, 1.f + e);
}
__device__ __forceinline__ float gate_act(int act, float g) {
  if (act == FLCE_ACT_NONE) return g;
  return act == FLCE_ACT_SIGMOID ? sigmoid_of(g, expf(-fabsf(g))) : tanhf(g);
}
__device__ __forceinline__ float gate_slope(int act, float a) {
  if (act == FLCE_ACT_SIGMOID) return a * (1.f - a);
  return act == FLCE_ACT_TANH ? 1.f - a * a : 1.f;
}
// Of gates per element.  BF16: the rows that leave all have that type, and the exponential may be
// off by 2 + 1.2 |g| units of fp32, 105 at most where it is a normal number: 2^-16 of the sigmoid,
// 1/256 of half a step of what is stored; in sums over tokens, beside gates near 1, it comes to
// half a unit, since |g| exp(-|g|) is 0.37 at most.  65536 x 4096 in bf16, sigmoids: 401 us
// forward and 641 backward; 424 and 692 with expf.
template <bool BF16>
__device__ __forceinline__ Oct gate_act_each(int act, Oct g) {
  if (act == FLCE_ACT_SIGMOID) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = g.p[i];
      g.p[i] = BF16 ? make_float2(sigmoid_of(v.x, __expf(-fabsf(v.x))),
                                  sigmoid_of(v.y, __expf(-fabsf(v.y))))
                    : make_float2(gate_act(act, v.x), gate_act(act, v.y));
    }
  } else if (act == FLCE_ACT_TANH) {
#pragma unroll
    for (int i = 0; i < 4; ++i) g.p[i] = make_float2(tanhf(g.p[i].x), tanhf(g.p[i].y));
  }
  return g;
}
// Slopes of a pair without a branch, which would wait for loads in flight: a - a^2 and
// 1 - a^2 by their coefficients, or 1.
struct GateSlope {
  float c0, c1;
  bool one;
  __device__ __forceinline__ explicit GateSlope(int act)
      : c0(act == FLCE_ACT_TANH ? 1.f : 0.f),
        c1(act == FLCE_ACT_SIGMOID ? 1.f : 0.f),
        one(act == FLCE_ACT_NONE) {}
  __device__ __forceinline__ float2 operator()(float2 a) const {
    const float2 s = mad2(a, plus2(pair(c1), mul2(a, pair(-1.f))), pair(c0));
    return make_float2(one ? 1.f : s.x, one ? 1.f : s.y);
  }
};
// The same out of line, for what is done once: the code around it stays short.
static __device__ __noinline__ Oct gate_act_oct(int act, Oct g) {
  return gate_act_each<false>(act, g);
}

}  // namespace flce
