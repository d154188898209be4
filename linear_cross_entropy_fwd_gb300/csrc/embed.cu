// embed.cu -- embedding lookup with a scale, and its gradient.
//
//   forward    Y[i] = s * W[id_i]                     (0 where id_i is ignored)
//   backward   dW[v] (+)= s * sum_{i : id_i = v} dY[i]
//
// The forward pass and the sums are bound by memory traffic: one multiply or
// add per element.
//
// The gradient sums equal ids in fp32 in a fixed order (ascending tokens in a piece of
// a run, then the pieces), and gives the same bits on every run: no element of dW is
// added to twice.  Three launches:
//   1  sort     tokens by id, stable (radix digits of at most 9 bits), in one
//               launch: one CTA with everything in shared memory for up to
//               2048 tokens (7 to 13 us; at 4096 21 us against the cluster's
//               13), else one 8-CTA cluster, whose phases need only a cluster
//               barrier between them (14 us at 8192 tokens, 46 at 65536).  When
//               64 MB or more are cleared meanwhile, one CTA up to 4096 tokens:
//               the clearing takes as long, and runs on all other SMs (128 MB
//               in 19 us, against 23 beside a cluster).  The other CTAs of the
//               launch clear dW meanwhile when it is overwritten (a large one
//               in part: see kClearSplit); when it is added to, they fetch the
//               tokens' rows of it into L2 (8192 tokens of 4096 bf16 on a tied
//               weight: 60 -> 56 us; fetching dY instead changes nothing).
//   2  sum      a run of one id is cut into pieces of at most L entries; CTA c
//               adds up the pieces that begin in entries [c*C, (c+1)*C) of the
//               sorted order.  A run of one piece goes straight to dW; the
//               pieces of a longer one leave fp32 partial rows, and the run
//               goes on a list.  Further CTAs clear what the sort had no time
//               for, except the rows that have tokens.
//   3  join     adds the partial rows of each run on the list, in order.
#include <cmath>

#include "host_util.h"
#include "sm103.cuh"

namespace flce {
namespace {

struct Ids {
  const void* p;
  int32_t is32;
  __device__ int64_t operator[](int64_t i) const {
    return is32 ? static_cast<int64_t>(static_cast<const int32_t*>(p)[i])
                : static_cast<const int64_t*>(p)[i];
  }
};

// ------------------------------------------------------------------ forward
// One 16-byte vector: 8 bf16 or 4 fp32 elements, scaled in fp32 and rounded
// once (to nearest even) for bf16.
template <int ELT>
__device__ __forceinline__ uint4 scale_vec(uint4 v, float s) {
  if (ELT == 4) {
    v.x = __float_as_uint(__uint_as_float(v.x) * s);
    v.y = __float_as_uint(__uint_as_float(v.y) * s);
    v.z = __float_as_uint(__uint_as_float(v.z) * s);
    v.w = __float_as_uint(__uint_as_float(v.w) * s);
  } else {
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      w[k] = pack_bf16x2(__uint_as_float(w[k] << 16) * s,
                         __uint_as_float(w[k] & 0xffff0000u) * s);
  }
  return v;
}

constexpr int kFwdThreads = 256;
constexpr int kFwdVecs = 4;  // 16-byte loads in flight per thread

// Vector f of the output is vector f % nv of token f / nv.  The output is
// written once and not read here, so it leaves L2 first; table rows stay.
// INDEX: 32 bits unless the output has 2^31 vectors or more (65536 tokens of 4096
// bf16: 113 us, 6.3 TB/s of rows read once and written; with 64-bit divisions
// 121).
template <int ELT, class INDEX>
__global__ void __launch_bounds__(kFwdThreads)
    embed_fwd_kernel(const uint4* __restrict__ W, Ids ids, uint4* __restrict__ Y, int64_t total,
                     uint32_t nv, int64_t V, int64_t ignore_index, float scale, int32_t* status) {
  const INDEX base = static_cast<INDEX>(blockIdx.x) * (kFwdThreads * kFwdVecs) + threadIdx.x;
  uint4 v[kFwdVecs];
#pragma unroll
  for (int k = 0; k < kFwdVecs; ++k) {
    const INDEX f = base + k * kFwdThreads;
    v[k] = make_uint4(0u, 0u, 0u, 0u);
    if (f < total) {
      const INDEX i = f / nv;
      const uint32_t c = static_cast<uint32_t>(f - i * nv);
      const int64_t id = ids[i];
      if (id != ignore_index) {
        if (id >= 0 && id < V)
          v[k] = __ldg(W + id * nv + c);
        else if (status && c == 0)
          atomicOr(status, FLCE_DEV_TARGET);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kFwdVecs; ++k) {
    const INDEX f = base + k * kFwdThreads;
    if (f < total) __stcs(Y + f, scale_vec<ELT>(v[k], scale));
  }
}

template <int ELT>
void launch_fwd(const void* W, const Ids& ids, void* Y, int64_t total, uint32_t nv, int64_t V,
                int64_t ignore_index, float scale, int32_t* status, unsigned blocks,
                cudaStream_t s) {
  const uint4* w = static_cast<const uint4*>(W);
  uint4* y = static_cast<uint4*>(Y);
  if (total < (int64_t{1} << 31))
    embed_fwd_kernel<ELT, uint32_t><<<blocks, kFwdThreads, 0, s>>>(w, ids, y, total, nv, V,
                                                                   ignore_index, scale, status);
  else
    embed_fwd_kernel<ELT, int64_t><<<blocks, kFwdThreads, 0, s>>>(w, ids, y, total, nv, V,
                                                                  ignore_index, scale, status);
}

// --------------------------------------------------------------------- sort
constexpr int kSortCtas = 8;           // of the cluster, for more tokens than one CTA holds
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxDigitBits = 9;
constexpr int kMaxDigits = 1 << kMaxDigitBits;
constexpr int kOneCtaTokens = 4096;  // that fit
constexpr int kOneCtaFaster = 2048;
constexpr int64_t kClearHides = int64_t{64} << 20;
// A dW of this many bytes and more is cleared in two parts: what the sort has time
// for beside it (5.5 MB per us), the rest beside the sums, there without the rows that
// have tokens.  8192 tokens, 262 MB: 68 -> 60 us; 2.1 GB: 342 -> 310 (8 tokens: 332 ->
// 284); but 3001 tokens, 128 MB: 35.5 -> 38.4, the sums of which it slows down.
constexpr int64_t kClearSplit = int64_t{192} << 20;
constexpr int64_t kClearBase = int64_t{40} << 20;
constexpr int64_t kClearPerToken = 3 << 10;
constexpr int64_t kFetchMost = int64_t{128} << 20;  // bytes of rows, with repetitions
constexpr int64_t kFetchPiece = 1024;
constexpr int kHistBytes = (kSortWarps * kMaxDigits + 2 * kMaxDigits + 32) * 4;

// Shared memory of the sort: one CTA keeps the (key, token) pairs twice.
constexpr int sort_smem(int ctas) { return kHistBytes + (ctas == 1 ? kOneCtaTokens * 16 : 0); }

struct SortParams {
  Ids ids;
  int64_t N;               // < 2^31
  int64_t V;
  int64_t ignore_index;
  uint2* pair[2];          // [N] (key, token): scratch of the cluster's passes
  uint32_t* key;           // [N] sorted
  uint32_t* pos;           // [N] the tokens in that order
  uint32_t* counts;        // [0] tokens that take part, [1] runs to join
  float4* clear;           // dW, to be cleared (or NULL)
  int64_t clear_vecs;
  const uint8_t* fetch;    // dW, whose rows of the first
  int64_t fetch_tokens;    // so many tokens go into L2 meanwhile
  int64_t fetch_row;       // bytes of a row
  int32_t passes, digit_bits;
  int32_t* status;
};

// Exclusive prefix sum of one value per thread over the CTA.
__device__ uint32_t cta_exclusive_sum(uint32_t x, uint32_t* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    const uint32_t w = warp_sums[lane];
    uint32_t winc = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, winc, o);
      if (lane >= o) winc += y;
    }
    warp_sums[lane] = winc - w;
  }
  __syncthreads();
  return warp_sums[warp] + inc - x;
}

__device__ __forceinline__ uint32_t ld_shared_cluster_u32(uint32_t cluster_addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_addr) : "memory");
  return v;
}

// The lanes whose digit (of `bits` bits) is this lane's; `in`: whether the lane
// has one.  One ballot per bit.
__device__ __forceinline__ uint32_t same_digit(uint32_t d, int bits, bool in) {
  uint32_t peers = __ballot_sync(0xffffffffu, in);
#pragma unroll
  for (int b = 0; b < kMaxDigitBits; ++b) {
    if (b < bits) {
      const uint32_t m = __ballot_sync(0xffffffffu, (d >> b) & 1u);
      peers &= (d >> b) & 1u ? m : ~m;
    }
  }
  return peers;
}

// Least-significant-digit radix sort.  A warp owns a contiguous range of the
// entries, and warps are ordered by (CTA rank, warp), so placing each warp's
// entries in order after all earlier warps' entries of the same digit keeps
// equal digits in input order (stable).  Ignored and bad ids get the key V,
// which sorts behind every row.
template <int CTAS>
__global__ void __launch_bounds__(kSortThreads, 1) embed_sort_kernel(const SortParams p) {
  grid_launch_dependents();
  if (blockIdx.x >= CTAS) {  // not the sorting CTAs
    // rows of dW that will be added to, on their way into L2
    const int64_t warps = static_cast<int64_t>(gridDim.x - CTAS) * kSortWarps;
    for (int64_t i = static_cast<int64_t>(blockIdx.x - CTAS) * kSortWarps + (threadIdx.x >> 5);
         i < p.fetch_tokens; i += warps) {
      const int64_t id = p.ids[i];
      if (id < 0 || id >= p.V || id == p.ignore_index) continue;
      const uint8_t* row = p.fetch + id * p.fetch_row;
      for (int64_t at = (threadIdx.x & 31) * int64_t{kFetchPiece}; at < p.fetch_row;
           at += 32 * kFetchPiece) {
        const int64_t left = p.fetch_row - at;
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(row + at),
                     "r"(static_cast<uint32_t>(left < kFetchPiece ? left : kFetchPiece))
                     : "memory");
      }
    }
    const int64_t step = static_cast<int64_t>(gridDim.x - CTAS) * kSortThreads;
#pragma unroll 4
    for (int64_t i = static_cast<int64_t>(blockIdx.x - CTAS) * kSortThreads + threadIdx.x;
         i < p.clear_vecs; i += step)
      __stcs(p.clear + i, make_float4(0.f, 0.f, 0.f, 0.f));
    return;
  }
  extern __shared__ uint32_t sm[];
  uint32_t* hist = sm;                                // [warp][digit]
  uint32_t* total = sm + kSortWarps * kMaxDigits;     // [digit] this CTA's count
  uint32_t* base = total + kMaxDigits;                // [digit] first place of this CTA
  uint32_t* warp_sums = base + kMaxDigits;
  uint2* own = reinterpret_cast<uint2*>(warp_sums + 32);  // CTAS == 1: two lists of pairs
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = CTAS > 1 ? cluster_ctarank() : 0u;
  const uint32_t gwarp = rank * kSortWarps + warp;
  const int64_t per_warp = (p.N + CTAS * kSortWarps - 1) / (CTAS * kSortWarps);
  const int64_t lo = gwarp * per_warp < p.N ? gwarp * per_warp : p.N;
  const int64_t hi = lo + per_warp < p.N ? lo + per_warp : p.N;
  const uint32_t digits = 1u << p.digit_bits;
  uint32_t taking_part = 0u;  // of this warp's tokens
  if (rank == 0 && tid < 2) p.counts[tid] = 0u;

  for (int pass = 0; pass < p.passes; ++pass) {
    const int shift = pass * p.digit_bits;
    const bool odd = pass & 1;
    uint2* in = CTAS > 1 ? (odd ? p.pair[1] : p.pair[0]) : own + odd * kOneCtaTokens;
    uint2* out = CTAS > 1 ? (odd ? p.pair[0] : p.pair[1]) : own + !odd * kOneCtaTokens;
    for (uint32_t d = lane; d < digits; d += 32) hist[warp * kMaxDigits + d] = 0u;
    __syncwarp();
    // count (each warp owns its row of the histogram)
    for (int64_t i0 = lo; i0 < hi; i0 += 32) {
      const int64_t i = i0 + lane;
      uint32_t d = 0xffffffffu;
      bool part = false;
      if (i < hi) {
        uint32_t k;
        if (pass == 0) {
          const int64_t id = p.ids[i];
          part = id >= 0 && id < p.V && id != p.ignore_index;
          if (!part && id != p.ignore_index && p.status) atomicOr(p.status, FLCE_DEV_TARGET);
          k = part ? static_cast<uint32_t>(id) : static_cast<uint32_t>(p.V);
          in[i] = make_uint2(k, static_cast<uint32_t>(i));
        } else {
          k = CTAS > 1 ? __ldcg(&in[i].x) : in[i].x;
        }
        d = (k >> shift) & (digits - 1);
      }
      if (pass == 0) taking_part += __popc(__ballot_sync(0xffffffffu, part));
      const uint32_t peers = same_digit(d, p.digit_bits, i < hi);
      if (i < hi && lane == __ffs(peers) - 1) hist[warp * kMaxDigits + d] += __popc(peers);
      __syncwarp();
    }
    __syncthreads();
    // per digit: offsets of the warps within the CTA, and the CTA's count
    uint32_t mine = 0u;
    if (tid < static_cast<int>(digits)) {
#pragma unroll 8
      for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t c = hist[w * kMaxDigits + tid];
        hist[w * kMaxDigits + tid] = mine;
        mine += c;
      }
      if (CTAS > 1) total[tid] = mine;
    }
    uint32_t all = mine, before = 0u;
    if (CTAS > 1) {
      cluster_sync();
      if (tid < static_cast<int>(digits)) {
        const uint32_t a = smem_addr(&total[tid]);
        all = 0u;
#pragma unroll
        for (int r = 0; r < CTAS; ++r) {
          const uint32_t c = ld_shared_cluster_u32(mapa_shared(a, static_cast<uint32_t>(r)));
          if (r < static_cast<int>(rank)) before += c;
          all += c;
        }
      }
    }
    const uint32_t first = cta_exclusive_sum(all, warp_sums);
    if (tid < static_cast<int>(digits)) base[tid] = first + before;
    __syncthreads();
    // counts[0] was cleared before the barriers just passed
    if (pass == 0 && lane == 0 && taking_part) atomicAdd(p.counts, taking_part);
    // place
    const bool last = pass == p.passes - 1;
    for (int64_t i0 = lo; i0 < hi; i0 += 32) {
      const int64_t i = i0 + lane;
      uint32_t d = 0xffffffffu;
      uint2 e = make_uint2(0u, 0u);
      if (i < hi) {
        e = CTAS > 1 ? __ldcg(in + i) : in[i];
        d = (e.x >> shift) & (digits - 1);
      }
      const uint32_t peers = same_digit(d, p.digit_bits, i < hi);
      if (i < hi) {
        const uint32_t at = base[d] + hist[warp * kMaxDigits + d] +
                            __popc(peers & ((1u << lane) - 1u));
        if (last) {
          p.key[at] = e.x;
          p.pos[at] = e.y;
        } else {
          out[at] = e;
        }
      }
      __syncwarp();
      if (i < hi && lane == __ffs(peers) - 1) hist[warp * kMaxDigits + d] += __popc(peers);
      __syncwarp();
    }
    // this pass's entries are in place, and every `total` has been read
    if (CTAS > 1)
      cluster_sync();
    else
      __syncthreads();
  }
}

// ---------------------------------------------------------------------- sum
constexpr int kSumThreads = 256;  // at most: one per 16-byte vector of a row
constexpr int kAhead = 8;         // rows in flight
constexpr int kMaxChunk = 64;
constexpr int kMinPiece = 32;
constexpr int kMaxPiece = kMaxChunk;  // pieces are at least as long as chunks
constexpr int64_t kClearUnit = int64_t{256} << 10;  // bytes that a CTA clears, at least one row
constexpr int kMaxClearRows = 1024;

struct SumParams {
  const void* dY;
  const uint32_t* key;       // sorted
  const uint32_t* pos;
  uint32_t* counts;          // see SortParams
  uint2* runs;               // [chunks] runs to join: first entry and id
  float* dW;
  float* partial;            // [chunks][2][H]: the last piece of a run; any other piece
  int64_t H, V;
  uint32_t nv;               // 16-byte vectors of dY per row
  int32_t chunk;             // C: entries per CTA
  int32_t piece;             // L >= C
  int32_t chunks;
  int32_t accumulate;
  float scale;
  int64_t clear_from;        // rows [clear_from, V) that no token has are cleared here,
  int32_t clear_rows;        // so many rows per CTA
};

// The first of the sorted entries [lo, hi) whose key is not less than k, or hi
// (the whole CTA): every round probes one place per thread.
__device__ __forceinline__ int64_t first_not_less(const uint32_t* key, int64_t lo, int64_t hi,
                                                  uint32_t k) {
  const int threads = static_cast<int>(blockDim.x);
  while (lo < hi) {
    const int64_t step = (hi - lo + threads - 1) / threads;
    const int64_t i = lo + threadIdx.x * step;
    const int less = __syncthreads_count(i < hi && __ldcg(key + i) < k);
    const int64_t top = lo + less * step;  // the first probe that is not less, or past them
    if (top < hi) hi = top;
    if (less > 0) lo = lo + (less - 1) * step + 1;
  }
  return hi;
}

// Clears those of a unit's rows that no token has.
__device__ void clear_unit(const SumParams& p, int64_t unit) {
  __shared__ uint32_t s_has[kMaxClearRows / 32];  // rows with tokens
  const int threads = static_cast<int>(blockDim.x);
  const int64_t n = p.counts[0];
  const int64_t a = p.clear_from + unit * p.clear_rows;
  if (a >= p.V) return;
  const int64_t b = a + p.clear_rows < p.V ? a + p.clear_rows : p.V;
  for (int i = threadIdx.x; i < kMaxClearRows / 32; i += threads) s_has[i] = 0u;
  int64_t i = first_not_less(p.key, 0, n, static_cast<uint32_t>(a)) + threadIdx.x;
  __syncthreads();
  for (;; i += threads) {
    const uint32_t k = i < n ? __ldcg(p.key + i) : 0xffffffffu;
    const bool in = k < static_cast<uint32_t>(b);  // b <= V < 2^31
    if (in) atomicOr(&s_has[(k - a) >> 5], 1u << ((k - a) & 31));
    if (!__syncthreads_or(in)) break;
  }
  const uint32_t h4 = static_cast<uint32_t>(p.H / 4);
  const uint32_t vecs = static_cast<uint32_t>(b - a) * h4;  // kClearUnit / 16, or one row
  float4* dst = reinterpret_cast<float4*>(p.dW + a * p.H);
#pragma unroll 4
  for (uint32_t v = threadIdx.x; v < vecs; v += threads) {
    const uint32_t r = v / h4;
    if (!((s_has[r >> 5] >> (r & 31)) & 1u)) __stcs(dst + v, make_float4(0.f, 0.f, 0.f, 0.f));
  }
}

template <int ELT>
struct Acc {  // the elements of one 16-byte vector in fp32
  static constexpr int kN = 16 / ELT;
  float a[kN];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int k = 0; k < kN; ++k) a[k] = 0.f;
  }
  __device__ __forceinline__ void add(const uint4& v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (ELT == 4) {
        a[k] += __uint_as_float(w[k]);
      } else {
        a[2 * k] += __uint_as_float(w[k] << 16);
        a[2 * k + 1] += __uint_as_float(w[k] & 0xffff0000u);
      }
    }
  }
  __device__ __forceinline__ void put(float* dst) const {  // as is
#pragma unroll
    for (int k = 0; k < kN; k += 4)
      *reinterpret_cast<float4*>(dst + k) = make_float4(a[k], a[k + 1], a[k + 2], a[k + 3]);
  }
};

// dW row piece: (dW +) scale * sum.  The addition is done at L2, so that no
// thread waits for the old value; every element gets one addend.  (L2 takes subnormal
// numbers for zeros.)
__device__ __forceinline__ void finish4(float* dst, float4 v, float scale, bool accumulate) {
  v.x *= scale;
  v.y *= scale;
  v.z *= scale;
  v.w *= scale;
  if (accumulate)
    asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(dst), "f"(v.x), "f"(v.y),
                 "f"(v.z), "f"(v.w)
                 : "memory");
  else
    *reinterpret_cast<float4*>(dst) = v;
}

// Grid: x = chunks, y = slices of the row.  Since L >= C, at most one piece
// that does not end its run begins in a chunk, and at most one that ends a run
// begun earlier: two partial rows per chunk hold whatever a chunk leaves.
template <int ELT>
__global__ void __launch_bounds__(kSumThreads) embed_sum_kernel(const SumParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t chunk = blockIdx.x;
  if (chunk >= p.chunks) {
    clear_unit(p, (chunk - p.chunks) * gridDim.y + blockIdx.y);
    return;
  }
  __shared__ uint32_t s_key[kMaxChunk + kMaxPiece + 2];  // entry i0 - 1 + t at t
  __shared__ uint32_t s_pos[kMaxChunk + kMaxPiece];
  const int64_t n = p.counts[0];
  const int C = p.chunk, L = p.piece, threads = static_cast<int>(blockDim.x);
  const int64_t i0 = chunk * C;
  if (i0 >= n) return;
  const int cnt = static_cast<int>(n - i0 < C + L ? n - i0 : C + L);  // entries in reach
  constexpr uint32_t kNone = 0xffffffffu;  // no row has this id (ids < 2^31)
  for (int t = threadIdx.x; t < cnt + 2; t += threads) {
    const int64_t i = i0 + t - 1;
    s_key[t] = (i >= 0 && i < n) ? __ldcg(p.key + i) : kNone;
    if (t >= 1 && t <= cnt) s_pos[t - 1] = __ldcg(p.pos + i);
  }
  __syncthreads();
  const uint32_t* key = s_key + 1;
  int j = 0;            // first entry of the next piece
  bool first = true;    // it begins its run
  if (key[-1] == key[0]) {
    // the run began earlier: how much earlier decides where its pieces begin
    const uint32_t k0 = key[0];
    const int64_t back = i0 - first_not_less(p.key, 0, i0 - 1, k0);
    const int next = static_cast<int>((L - back % L) % L);
    while (j < next && j < cnt && key[j] == k0) ++j;
    first = !(j < cnt && key[j] == k0);
  }
  const uint4* dY = static_cast<const uint4*>(p.dY);
  const uint32_t c = blockIdx.y * threads + threadIdx.x;  // vector of the row
  if (c >= p.nv) return;
  constexpr int kN = Acc<ELT>::kN;
  Acc<ELT> acc;
  acc.zero();
  int from = j;  // first entry of the current piece
  bool done = j >= C || j >= cnt;
  while (!done) {
    uint4 v[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a)
      if (j + a < cnt) v[a] = __ldcs(dY + static_cast<int64_t>(s_pos[j + a]) * p.nv + c);
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      if (done) break;
      acc.add(v[a]);
      const uint32_t k = key[j];
      ++j;
      const bool goes_on = key[j] == k;  // key[cnt] is in place too
      if (goes_on && j - from < L) continue;
      if (goes_on && first && c == 0)
        p.runs[atomicAdd(p.counts + 1, 1u)] =  // in any order: the runs are disjoint
            make_uint2(static_cast<uint32_t>(i0 + from), k);
      if (!first || goes_on) {
        const int64_t slot = 2 * chunk + (goes_on ? 1 : 0);
        acc.put(p.partial + slot * p.H + static_cast<int64_t>(c) * kN);
      } else {
        float* dst = p.dW + static_cast<int64_t>(k) * p.H + static_cast<int64_t>(c) * kN;
#pragma unroll
        for (int e = 0; e < kN; e += 4)
          finish4(dst + e, make_float4(acc.a[e], acc.a[e + 1], acc.a[e + 2], acc.a[e + 3]),
                   p.scale, p.accumulate != 0);
      }
      acc.zero();
      first = !goes_on;
      from = j;
      done = j >= C || j >= cnt;
    }
  }
}

// --------------------------------------------------------------------- join
// One work item per (run on the list, slice of the row).  The pieces of a run
// that begins at entry r begin at r, r + L, r + 2 L, ...; each left its sum with
// the chunk it begins in.  Eight groups of threads take contiguous shares of
// the pieces; their sums are added in order.
constexpr int kJoinCols = 32;    // float4 columns per item
constexpr int kJoinGroups = 8;
constexpr int kJoinThreads = kJoinCols * kJoinGroups;

__global__ void __launch_bounds__(kJoinThreads) embed_join_kernel(const SumParams p) {
  grid_dependency_wait();
  __shared__ float4 s_part[kJoinGroups][kJoinCols];
  const int64_t n = p.counts[0];
  const int64_t C = p.chunk, L = p.piece;
  const int64_t h4 = p.H / 4;
  const int64_t slices = (h4 + kJoinCols - 1) / kJoinCols;
  const int64_t items = p.counts[1] * slices;
  const float4* part = reinterpret_cast<const float4*>(p.partial);
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const uint2 run = __ldcg(p.runs + item / slices);
    const int64_t r = run.x;
    const uint32_t k = run.y;
    int64_t pieces = 0;
    for (;;) {
      const int64_t e = r + (pieces + threadIdx.x) * L;
      const int hit = __syncthreads_count(e < n && __ldcg(p.key + e) == k);
      pieces += hit;
      if (hit < kJoinThreads) break;
    }
    const int group = threadIdx.x / kJoinCols, col = threadIdx.x % kJoinCols;
    const int64_t x = item % slices * kJoinCols + col;
    const int64_t share = (pieces + kJoinGroups - 1) / kJoinGroups;
    const int64_t lo = group * share;
    const int64_t hi = lo + share < pieces ? lo + share : pieces;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (x < h4) {
#pragma unroll 8
      for (int64_t q = lo; q < hi; ++q) {
        const int64_t slot = 2 * ((r + q * L) / C) + (q + 1 < pieces ? 1 : 0);
        const float4 v = __ldcs(part + slot * h4 + x);
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
      }
    }
    s_part[group][col] = s;
    __syncthreads();
    if (group == 0 && x < h4) {
#pragma unroll
      for (int g = 1; g < kJoinGroups; ++g) {
        const float4 v = s_part[g][col];
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
      }
      finish4(p.dW + static_cast<int64_t>(k) * p.H + 4 * x, s, p.scale, p.accumulate != 0);
    }
  }  // the next item's barrier comes before s_part is written again
}

// --------------------------------------------------------------------- host
int check_embed(const char* who, const void* table, const void* rows, const void* ids, int64_t N,
                int64_t H, int64_t V, float scale, int32_t dtype) {
  if (dtype != FLCE_BF16 && dtype != FLCE_FP32)
    return host_error(FLCE_ERR_ARG, "%s: unknown dtype %d", who, dtype);
  if (N < 0 || H <= 0 || V <= 0 || N >= (int64_t{1} << 31) || V >= (int64_t{1} << 31) ||
      H > (int64_t{1} << 20))
    return host_error(FLCE_ERR_ARG,
                      "%s: sizes must satisfy 0 <= N < 2^31, 0 < H <= 2^20, 0 < V < 2^31", who);
  if (!table || (N > 0 && (!rows || !ids)))
    return host_error(FLCE_ERR_ARG, "%s: null pointer", who);
  // (an infinite scale would make NaN of the zeros that ignored tokens get)
  if (!std::isfinite(scale)) return host_error(FLCE_ERR_ARG, "%s: scale must be finite", who);
  const int elt = dtype == FLCE_FP32 ? 4 : 2;
  if ((H * elt) % 16 != 0)
    return host_error(FLCE_ERR_ALIGN, "%s: H * sizeof(element) = %lld is not a multiple of 16",
                      who, static_cast<long long>(H * elt));
  if (!aligned16(table) || !aligned16(rows))
    return host_error(FLCE_ERR_ALIGN, "%s: buffers must be 16-byte aligned", who);
  return FLCE_OK;
}

bool one_cta_sorts(int64_t N, int64_t clear_bytes) {
  return N <= kOneCtaFaster || (N <= kOneCtaTokens && clear_bytes >= kClearHides);
}

struct BwdPlan {
  int32_t passes, digit_bits, chunk, piece, chunks;
  size_t key, pos, pair[2], counts, runs, partial, total;
};

// Entries per CTA of the sum: enough CTAs for twelve on each of 152 SMs,
// within 4 .. kMaxChunk.
BwdPlan plan_bwd(int64_t N, int64_t H, int64_t V, int elt, bool one_cta) {
  BwdPlan b{};
  int bits = 1;
  while ((int64_t{1} << bits) <= V) ++bits;  // keys 0 .. V
  b.passes = (bits + kMaxDigitBits - 1) / kMaxDigitBits;
  b.digit_bits = (bits + b.passes - 1) / b.passes;
  const int64_t slices = (H * elt / 16 + kSumThreads - 1) / kSumThreads;
  int64_t c = (N * slices + 152 * 12 - 1) / (152 * 12);
  if (c < 4) c = 4;
  if (c > kMaxChunk) c = kMaxChunk;
  b.chunk = static_cast<int32_t>(c);
  b.piece = b.chunk > kMinPiece ? b.chunk : kMinPiece;
  b.chunks = static_cast<int32_t>((N + c - 1) / c);
  size_t o = 0;
  const size_t list = round256(static_cast<size_t>(N) * 4);
  b.key = o;
  o += list;
  b.pos = o;
  o += list;
  for (int i = 0; i < 2; ++i) {
    b.pair[i] = o;
    if (!one_cta) o += round256(static_cast<size_t>(N) * 8);
  }
  b.counts = o;
  o += 256;
  b.runs = o;
  o += round256(static_cast<size_t>(b.chunks) * 8);
  b.partial = o;
  o += round256(static_cast<size_t>(b.chunks) * 2 * static_cast<size_t>(H) * 4);
  b.total = o;
  return b;
}

// A launch whose CTAs may start while the previous launch finishes; the kernel
// waits for it before it reads.
template <class KernelT, class P>
cudaError_t launch_after(KernelT kernel, dim3 grid, int threads, const P& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int CTAS>
cudaError_t launch_sort(const SortParams& p, int sms, cudaStream_t s) {
  static SmemLimit limit;
  const cudaError_t e = limit.raise(embed_sort_kernel<CTAS>, sort_smem(CTAS));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  // the sorting CTAs, and others that clear and fetch: one on each of the other
  // SMs, or 14 clusters, which find room beside the sorting one
  cfg.gridDim = dim3(static_cast<unsigned>(CTAS + (CTAS == 1 ? sms - 1 : 14 * CTAS)));
  cfg.blockDim = dim3(kSortThreads);
  cfg.dynamicSmemBytes = sort_smem(CTAS);
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CTAS;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, embed_sort_kernel<CTAS>, p);
}

int run_bwd(const SortParams& sort, const SumParams& sum, int elt, bool one_cta, int sms,
            cudaStream_t s) {
  FLCE_TRY(one_cta ? launch_sort<1>(sort, sms, s) : launch_sort<kSortCtas>(sort, sms, s));
  const unsigned slices = (sum.nv + kSumThreads - 1) / kSumThreads;
  const int threads = static_cast<int>(((sum.nv + slices - 1) / slices + 31) / 32 * 32);
  int64_t x = sum.chunks;
  if (sum.clear_from < sum.V) {
    const int64_t units = (sum.V - sum.clear_from + sum.clear_rows - 1) / sum.clear_rows;
    x += (units + slices - 1) / slices;
  }
  const dim3 g(static_cast<unsigned>(x), slices);
  FLCE_TRY(elt == 2 ? launch_after(embed_sum_kernel<2>, g, threads, sum, s)
                    : launch_after(embed_sum_kernel<4>, g, threads, sum, s));
  if (sort.N > sum.piece)  // else no run is longer than a piece
    FLCE_TRY(launch_after(embed_join_kernel, dim3(static_cast<unsigned>(sms) * 4), kJoinThreads,
                          sum, s));
  return FLCE_OK;
}

}  // namespace
}  // namespace flce

using namespace flce;

extern "C" {

int flce_embed_fwd(const void* W, const void* ids, int64_t N, int64_t H, int64_t V, float scale,
                   int64_t ignore_index, void* Y, const flce_opts* opts) {
  host_clear_error();
  const flce_opts o = opts_or_default(opts);
  int rc = check_embed("flce_embed_fwd", W, Y, ids, N, H, V, scale, o.dtype);
  if (rc) return rc;
  int sms = 0;
  if ((rc = host_device(&sms))) return rc;
  StepCall call;
  if ((rc = call.begin(o, 0, StepCall::kIfAsked))) return rc;
  if (N > 0) {
    const int elt = o.dtype == FLCE_FP32 ? 4 : 2;
    const uint32_t nv = static_cast<uint32_t>(H * elt / 16);
    const int64_t total = N * nv;
    const int64_t blocks = (total + kFwdThreads * kFwdVecs - 1) / (kFwdThreads * kFwdVecs);
    const Ids id{ids, o.target_is_int32 != 0 ? 1 : 0};
    if (blocks > 0x7fffffff) {
      rc = host_error(FLCE_ERR_ARG, "flce_embed_fwd: N * H is too large for one call");
    } else {
      const unsigned g = static_cast<unsigned>(blocks);
      if (elt == 2)
        launch_fwd<2>(W, id, Y, total, nv, V, ignore_index, scale, call.status, g, call.stream);
      else
        launch_fwd<4>(W, id, Y, total, nv, V, ignore_index, scale, call.status, g, call.stream);
      const cudaError_t e = cudaGetLastError();
      if (e != cudaSuccess) rc = host_cuda_error(e, "embed_fwd");
    }
  }
  return call.end(rc);
}

int flce_embed_bwd(const void* dY, const void* ids, int64_t N, int64_t H, int64_t V, float scale,
                   int64_t ignore_index, float* dW, int32_t accumulate, const flce_opts* opts) {
  host_clear_error();
  const flce_opts o = opts_or_default(opts);
  int rc = check_embed("flce_embed_bwd", dW, dY, ids, N, H, V, scale, o.dtype);
  if (rc) return rc;
  int sms = 0;
  if ((rc = host_device(&sms))) return rc;
  const int elt = o.dtype == FLCE_FP32 ? 4 : 2;
  const int64_t beside_sort = (kClearBase + N * kClearPerToken) / (H * 4);
  const int64_t clear_first =
      accumulate ? 0 : V * H * 4 < kClearSplit || V < beside_sort ? V : beside_sort;
  const bool one_cta = one_cta_sorts(N, clear_first * H * 4);
  const BwdPlan b = plan_bwd(N, H, V, elt, one_cta);
  StepCall call;
  if ((rc = call.begin(o, N > 0 ? b.total : 0, StepCall::kIfAsked))) return rc;
  if (N == 0) {
    if (!accumulate) {
      const cudaError_t e =
          cudaMemsetAsync(dW, 0, static_cast<size_t>(V) * static_cast<size_t>(H) * 4, call.stream);
      if (e != cudaSuccess) rc = host_cuda_error(e, "cudaMemsetAsync(dW)");
    }
    return call.end(rc);
  }
  uint8_t* w = call.scratch;
  SortParams sp{};
  sp.ids = Ids{ids, o.target_is_int32 != 0 ? 1 : 0};
  sp.N = N;
  sp.V = V;
  sp.ignore_index = ignore_index;
  sp.key = reinterpret_cast<uint32_t*>(w + b.key);
  sp.pos = reinterpret_cast<uint32_t*>(w + b.pos);
  for (int i = 0; i < 2; ++i) sp.pair[i] = reinterpret_cast<uint2*>(w + b.pair[i]);
  sp.counts = reinterpret_cast<uint32_t*>(w + b.counts);
  sp.clear = accumulate ? nullptr : reinterpret_cast<float4*>(dW);
  sp.clear_vecs = clear_first * H / 4;
  sp.fetch = reinterpret_cast<const uint8_t*>(dW);
  sp.fetch_row = H * 4;
  const int64_t fetch = kFetchMost / sp.fetch_row;
  sp.fetch_tokens = accumulate ? (N < fetch ? N : fetch) : 0;
  sp.passes = b.passes;
  sp.digit_bits = b.digit_bits;
  sp.status = call.status;
  SumParams sm{};
  sm.dY = dY;
  sm.key = sp.key;
  sm.pos = sp.pos;
  sm.counts = sp.counts;
  sm.runs = reinterpret_cast<uint2*>(w + b.runs);
  sm.dW = dW;
  sm.partial = reinterpret_cast<float*>(w + b.partial);
  sm.H = H;
  sm.V = V;
  sm.nv = static_cast<uint32_t>(H * elt / 16);
  sm.chunk = b.chunk;
  sm.piece = b.piece;
  sm.chunks = b.chunks;
  sm.accumulate = accumulate != 0 ? 1 : 0;
  sm.scale = scale;
  sm.clear_from = accumulate ? V : clear_first;
  const int64_t rows = kClearUnit / (H * 4);
  sm.clear_rows = static_cast<int32_t>(rows < 1 ? 1 : rows > kMaxClearRows ? kMaxClearRows : rows);
  return call.end(run_bwd(sp, sm, elt, one_cta, sms, call.stream));
}

}  // extern "C"
