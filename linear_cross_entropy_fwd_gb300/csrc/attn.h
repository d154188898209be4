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
  AttnTile* tiles;      // [max_tiles] units, highest index first
  int32_t* n_tiles;
  int32_t* bucket;      // [max_depth + 2] scratch of the plan
  int32_t max_tiles;    // an upper bound from B and T alone
  int32_t max_depth;    // units of the longest possible sequence
  float* lse;           // [Hq][T]
  float* delta;         // [Hq][T]
  AttnOut o, dO, dq, dk, dv;
  int32_t* status;
};

// Launchers.  Tensor maps: box 64 x 1 x 128 of [T, heads, D], 128-byte swizzle.
cudaError_t launch_attn_plan(const AttnParams& p, bool backward, int sms, cudaStream_t s);
cudaError_t launch_attn_fwd(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                            const AttnParams& p, int sms, cudaStream_t s);
cudaError_t launch_attn_dkdv(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                             const CUtensorMap& dO, const AttnParams& p, int sms, cudaStream_t s);
cudaError_t launch_attn_dq(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                           const CUtensorMap& dO, const AttnParams& p, cudaStream_t s);

}  // namespace flce
