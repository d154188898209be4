// attn.h -- what the packed causal attention kernels and their host side
// share (internal).
//
// Sequences lie one after the other in [T] tokens: sequence b is tokens
// cu[b] .. cu[b+1]-1.  Within a sequence, for query head h and kv head
// h / (Hq / Hkv):
//   S = scale Q K^T,  S_ij = -inf for j > i
//   lse_i = ln sum_j exp S_ij,  P = exp(S - lse),  O = P V
//   delta_i = sum_d dO_id O_id,  dS = P o (dO V^T - delta)
//   dV = P^T dO,  dK = scale dS^T Q,  dQ = scale dS K
// (dV and dK summed over the query heads of the group).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

namespace flce {

constexpr int kTile = 128;  // rows of a query tile and of a key tile

// One unit of work of a sequence: `unit` consecutive tiles (AttnParams).
struct AttnTile {
  int32_t start;  // first token of the sequence
  int32_t len;    // its length
  int32_t tile;   // index of the unit within the sequence
  int32_t pad;
};

// Strides in elements of a [T, heads, D] tensor whose D axis is contiguous.
struct AttnOut {
  void* p;
  int64_t token, head;
};

struct AttnParams {
  const int32_t* cu;    // [B + 1]
  int32_t B, T, Hq, Hkv, D;
  float scale;          // > 0
  int32_t unit;         // tiles per unit: 2 forward, 1 backward
  AttnTile* tiles;      // [max_tiles] units, highest index first (NULL: no plan)
  int32_t* n_tiles;
  int32_t* bucket;      // [max_depth + 2] scratch of the plan
  int32_t max_tiles;    // an upper bound from B and T alone
  int32_t max_depth;    // units of the longest possible sequence
  float* lse;           // [Hq][T]
  float* delta;         // [Hq][T]
  AttnOut k, v, o, dO, dq, dk, dv;
  int32_t* status;      // may be NULL without a plan
};

// Zeros in the rows [t0, t1) of a [T, heads, D] output, 16 bytes at a time.
__device__ inline void zero_rows(const AttnOut& o, int heads, int D, int t0, int t1, int64_t me,
                          int64_t threads) {
  const int vecs = D / 8;
  const int64_t per = static_cast<int64_t>(heads) * vecs, n = (t1 - t0) * per;
  for (int64_t i = me; i < n; i += threads) {
    const int64_t t = t0 + i / per;
    const int r = static_cast<int>(i % per);
    uint4* d = reinterpret_cast<uint4*>(static_cast<uint16_t*>(o.p) + t * o.token +
                                        (r / vecs) * o.head + (r % vecs) * 8);
    *d = make_uint4(0u, 0u, 0u, 0u);
  }
}

// What the tokens before the first sequence and after the last get (all tokens
// if the offsets are bad): zeros, and an lse of -inf.
template <bool BACKWARD>
__device__ void blank_outside(const AttnParams& p, bool ok, int64_t me, int64_t threads) {
  const int lo = ok ? p.cu[0] : p.T, hi = ok ? p.cu[p.B] : p.T;
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    const int t0 = side ? hi : 0, t1 = side ? p.T : lo;
    if (t0 >= t1) continue;
    if (BACKWARD) {
      zero_rows(p.dq, p.Hq, p.D, t0, t1, me, threads);
      zero_rows(p.dk, p.Hkv, p.D, t0, t1, me, threads);
      zero_rows(p.dv, p.Hkv, p.D, t0, t1, me, threads);
    } else {
      zero_rows(p.o, p.Hq, p.D, t0, t1, me, threads);
      const int64_t n = static_cast<int64_t>(p.Hq) * (t1 - t0);
      for (int64_t i = me; i < n; i += threads)
        p.lse[i / (t1 - t0) * p.T + t0 + i % (t1 - t0)] = -INFINITY;
    }
  }
}

// A forward pass whose units all run at once has no plan: every CTA finds its own,
// with a thread per sequence (57, 1 and 130 tokens, 8 heads: 28 us with a plan, 19
// without on the same machine, most of it on the host; 18 to 27 us on others).
constexpr int kDirectSeqs = 256;

// Launchers.  Tensor maps: box 64 x 1 x 128 of [T, heads, D], 128-byte swizzle.
cudaError_t launch_attn_plan(const AttnParams& p, bool backward, int sms, cudaStream_t s);
cudaError_t launch_attn_fwd(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                            const AttnParams& p, int sms, cudaStream_t s);
cudaError_t launch_attn_dkdv(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                             const CUtensorMap& dO, const AttnParams& p, int sms, cudaStream_t s);
cudaError_t launch_attn_dq(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                           const CUtensorMap& dO, const AttnParams& p, cudaStream_t s);

}  // namespace flce
