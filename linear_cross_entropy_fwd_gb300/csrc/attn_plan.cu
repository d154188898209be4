// attn_plan.cu -- the first launch of an attention call (a small forward pass has
// none: see kDirectSeqs).  Block 0 turns the
// sequence offsets into the list of tiles, longest work first, so that the
// last CTAs to start are the short ones.  The other blocks write what no
// tile covers (tokens outside every sequence) and, for the backward pass,
// delta.
#include "attn.h"
#include "host_util.h"
#include "sm103.cuh"

namespace flce {
namespace {

constexpr int kThreads = 256;
constexpr int kSharedDepth = 4096;  // buckets kept in shared memory

// Whether 0 <= cu[0] <= ... <= cu[B] <= T (the same answer in every thread).
__device__ bool offsets_ok(const AttnParams& p) {
  int bad = 0;
  for (int b = threadIdx.x; b <= p.B; b += kThreads) {
    const int c = p.cu[b];
    bad |= (c < 0) || (c > p.T) || (b > 0 && c < p.cu[b - 1]);
  }
  return __syncthreads_or(bad) == 0;
}

// The units of a sequence meet the more tiles the higher their index (a key
// tile's, counted from the sequence's end).  Counting sort by that index, the
// highest first; units of one index come in any order.
__device__ void make_tiles(const AttnParams& p, bool ok) {
  __shared__ int32_t s_bucket[kSharedDepth];
  __shared__ int32_t s_warp[kThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) *p.status = ok ? 0 : FLCE_DEV_SEQLENS;  // clears it for this call
  if (!ok) {
    if (threadIdx.x == 0) *p.n_tiles = 0;
    return;
  }
  const int unit = kTile * p.unit;  // tokens
  int32_t* bucket = p.max_depth < kSharedDepth ? s_bucket : p.bucket;
  for (int k = threadIdx.x; k <= p.max_depth; k += kThreads) bucket[k] = 0;
  __syncthreads();
  for (int b = warp; b < p.B; b += kThreads / 32) {
    const int nt = (p.cu[b + 1] - p.cu[b] + unit - 1) / unit;
    for (int i = lane; i < nt; i += 32) atomicAdd(&bucket[i], 1);
  }
  __syncthreads();
  // bucket[k] = number of units of a higher index
  int32_t above = 0;
  for (int top = p.max_depth; top >= 0; top -= kThreads) {
    const int k = top - static_cast<int>(threadIdx.x);
    const int32_t c = k >= 0 ? bucket[k] : 0;
    int32_t inc = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    int32_t before = 0, all = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += s_warp[w];
      all += s_warp[w];
    }
    if (k >= 0) bucket[k] = above + before + inc - c;
    above += all;
    __syncthreads();
  }
  for (int b = warp; b < p.B; b += kThreads / 32) {
    const int c0 = p.cu[b], len = p.cu[b + 1] - c0;
    const int nt = (len + unit - 1) / unit;
    for (int i = lane; i < nt; i += 32) {
      const int at = atomicAdd(&bucket[i], 1);
      p.tiles[at] = AttnTile{c0, len, i, 0};
    }
  }
  if (threadIdx.x == 0) *p.n_tiles = above;
}

// delta of every token: 16 lanes per (head, token), eight products each.  It comes from
// the stored o, rounded to bf16 (o in fp32 would be twice the bytes to keep and read):
// of the gradients' error, 2.5e-3 of their norm in a batch of 2048 tokens, that is
// 0.9e-3, their own rounding and that of dS 1.7e-3 each.
__device__ void make_delta(const AttnParams& p, int64_t me, int64_t threads) {
  const int part = static_cast<int>(me & 15);
  const int64_t n = static_cast<int64_t>(p.Hq) * p.T;
  for (int64_t u = me >> 4; (u & ~int64_t{1}) < n; u += threads >> 4) {  // warp-uniform bound
    float s = 0.f;
    const int64_t h = u / p.T, t = u - h * p.T;
    if (u < n && part * 8 < p.D) {
      const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.o.p) +
                                                      t * p.o.token + h * p.o.head + part * 8);
      const uint4 b = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.dO.p) +
                                                      t * p.dO.token + h * p.dO.head + part * 8);
      const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        s = fmaf(__uint_as_float(x[k] << 16), __uint_as_float(y[k] << 16), s);
        s = fmaf(__uint_as_float(x[k] & 0xffff0000u), __uint_as_float(y[k] & 0xffff0000u), s);
      }
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (u < n && part == 0) p.delta[u] = s;
  }
}

template <bool BACKWARD>
__global__ void __launch_bounds__(kThreads) attn_plan_kernel(const AttnParams p) {
  grid_launch_dependents();  // the next launch's setup may overlap this one
  const bool ok = offsets_ok(p);
  if (blockIdx.x == 0) {
    make_tiles(p, ok);
    return;
  }
  const int64_t me = static_cast<int64_t>(blockIdx.x - 1) * kThreads + threadIdx.x;
  const int64_t threads = static_cast<int64_t>(gridDim.x - 1) * kThreads;
  blank_outside<BACKWARD>(p, ok, me, threads);
  if (BACKWARD) make_delta(p, me, threads);
}

}  // namespace

cudaError_t launch_attn_plan(const AttnParams& p, bool backward, int sms, cudaStream_t s) {
  // forward: little beside the list; backward: delta reads all of o and dO
  const int64_t want = (static_cast<int64_t>(p.Hq) * p.T + 15) / 16;
  const int64_t cap = backward ? static_cast<int64_t>(sms) * 8 : 16;
  const unsigned blocks = 1u + static_cast<unsigned>(want < cap ? (want < 1 ? 1 : want) : cap);
  if (backward)
    attn_plan_kernel<true><<<blocks, kThreads, 0, s>>>(p);
  else
    attn_plan_kernel<false><<<blocks, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace flce
