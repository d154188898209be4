// embed.cu -- embedding lookup with a scale, and its gradient.
//
//   forward    Y[i] = s * W[id_i]                     (0 where id_i is ignored)
//   backward   dW[v] (+)= s * sum_{i : id_i = v} dY[i]
//
// The forward pass and the sums are bound by memory traffic: one multiply or
// add per element.
//
// The gradient sums equal ids in ascending token order, in fp32, and gives
// the same bits on every run: no floating-point atomics.  Three launches:
//   1  sort     tokens by id, stable (one 8-CTA cluster, radix digits of at
//               most 9 bits).  One launch, because its phases need only a
//               cluster barrier between them.
//   2  sum      CTA c walks entries [c*C, (c+1)*C) of the sorted order and
//               adds up runs of one id.  A run inside the chunk goes straight
//               to dW; a run that crosses a chunk's border leaves an fp32
//               partial row.  When dW is overwritten, further CTAs of the same
//               launch write zeros to the rows no token has (a bitmap made by
//               the sort says which), so each row is written once.
//   3  join     adds the partial rows of each crossing run, in order.
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
template <int ELT>
__global__ void __launch_bounds__(kFwdThreads)
    embed_fwd_kernel(const uint4* __restrict__ W, Ids ids, uint4* __restrict__ Y, int64_t total,
                     uint32_t nv, int64_t V, int64_t ignore_index, float scale, int32_t* status) {
  const int64_t base = static_cast<int64_t>(blockIdx.x) * (kFwdThreads * kFwdVecs) + threadIdx.x;
  uint4 v[kFwdVecs];
#pragma unroll
  for (int k = 0; k < kFwdVecs; ++k) {
    const int64_t f = base + k * kFwdThreads;
    v[k] = make_uint4(0u, 0u, 0u, 0u);
    if (f < total) {
      const int64_t i = f / nv;
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
    const int64_t f = base + k * kFwdThreads;
    if (f < total) __stcs(Y + f, scale_vec<ELT>(v[k], scale));
  }
}

// --------------------------------------------------------------------- sort
constexpr int kSortCtas = 8;
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxDigitBits = 9;
constexpr int kMaxDigits = 1 << kMaxDigitBits;
constexpr int kSortSmem = (kSortWarps * kMaxDigits + 2 * kMaxDigits + 32) * 4;

struct SortParams {
  Ids ids;
  int64_t N;               // < 2^31
  int64_t V;
  int64_t ignore_index;
  uint32_t* key[2];        // [N] each; the last pass writes key[passes & 1]
  uint32_t* pos[2];
  uint32_t* bitmap;        // ceil(V / 32) words: rows that have a token (or NULL)
  uint32_t* n_sorted;      // tokens that take part
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
    uint32_t w = lane < kSortWarps ? warp_sums[lane] : 0u;
    uint32_t winc = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, winc, o);
      if (lane >= o) winc += y;
    }
    if (lane < kSortWarps) warp_sums[lane] = winc - w;
  }
  __syncthreads();
  const uint32_t r = warp_sums[warp] + inc - x;
  __syncthreads();
  return r;
}

__device__ __forceinline__ uint32_t ld_shared_cluster_u32(uint32_t cluster_addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_addr) : "memory");
  return v;
}

// Least-significant-digit radix sort.  Token i belongs to the warp whose
// contiguous range holds it, and warps are ordered by (CTA rank, warp), so
// placing each warp's tokens in order after all earlier warps' tokens of the
// same digit keeps equal digits in input order (stable).  Ignored and bad ids
// get the key V, which sorts behind every row.
__global__ void __cluster_dims__(kSortCtas, 1, 1) __launch_bounds__(kSortThreads, 1)
    embed_sort_kernel(const SortParams p) {
  extern __shared__ uint32_t sm[];
  uint32_t* hist = sm;                                // [warp][digit]
  uint32_t* total = sm + kSortWarps * kMaxDigits;     // [digit] this CTA's count
  uint32_t* base = total + kMaxDigits;                // [digit] first place of this CTA
  uint32_t* warp_sums = base + kMaxDigits;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_ctarank();
  const uint32_t gwarp = rank * kSortWarps + warp;
  const int64_t per_warp = (p.N + kSortCtas * kSortWarps - 1) / (kSortCtas * kSortWarps);
  const int64_t lo = gwarp * per_warp < p.N ? gwarp * per_warp : p.N;
  const int64_t hi = lo + per_warp < p.N ? lo + per_warp : p.N;
  const uint32_t digits = 1u << p.digit_bits;

  if (p.bitmap) {
    const int64_t words = (p.V + 31) / 32;
    for (int64_t w = rank * kSortThreads + tid; w < words; w += kSortCtas * kSortThreads)
      p.bitmap[w] = 0u;
  }
  if (rank == 0 && tid == 0) *p.n_sorted = 0u;

  for (int pass = 0; pass < p.passes; ++pass) {
    const int shift = pass * p.digit_bits;
    const uint32_t* key_in = p.key[pass & 1];
    const uint32_t* pos_in = p.pos[pass & 1];
    uint32_t* key_out = p.key[(pass + 1) & 1];
    uint32_t* pos_out = p.pos[(pass + 1) & 1];
    auto load = [&](int64_t i, uint32_t& k, uint32_t& q) {
      if (pass == 0) {
        const int64_t id = p.ids[i];
        const bool in = id >= 0 && id < p.V && id != p.ignore_index;
        k = in ? static_cast<uint32_t>(id) : static_cast<uint32_t>(p.V);
        q = static_cast<uint32_t>(i);
        return in || id == p.ignore_index;
      }
      k = __ldcg(key_in + i);
      q = __ldcg(pos_in + i);
      return true;
    };
    for (uint32_t d = lane; d < digits; d += 32) hist[warp * kMaxDigits + d] = 0u;
    __syncwarp();
    // count (each warp owns its row of the histogram)
    for (int64_t i0 = lo; i0 < hi; i0 += 32) {
      const int64_t i = i0 + lane;
      uint32_t d = 0xffffffffu;
      if (i < hi) {
        uint32_t k, q;
        if (!load(i, k, q) && p.status) atomicOr(p.status, FLCE_DEV_TARGET);
        d = (k >> shift) & (digits - 1);
      }
      const uint32_t peers = __match_any_sync(0xffffffffu, d);
      if (i < hi && lane == __ffs(peers) - 1) hist[warp * kMaxDigits + d] += __popc(peers);
      __syncwarp();
    }
    __syncthreads();
    // per digit: offsets of the warps within the CTA, and the CTA's count
    uint32_t mine = 0u;
    if (tid < static_cast<int>(digits)) {
      for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t c = hist[w * kMaxDigits + tid];
        hist[w * kMaxDigits + tid] = mine;
        mine += c;
      }
      total[tid] = mine;
    }
    cluster_sync();
    uint32_t all = 0u, before = 0u;
    if (tid < static_cast<int>(digits)) {
      const uint32_t a = smem_addr(&total[tid]);
#pragma unroll
      for (uint32_t r = 0; r < kSortCtas; ++r) {
        const uint32_t c = ld_shared_cluster_u32(mapa_shared(a, r));
        if (r < rank) before += c;
        all += c;
      }
    }
    const uint32_t first = cta_exclusive_sum(all, warp_sums);
    if (tid < static_cast<int>(digits)) base[tid] = first + before;
    __syncthreads();
    // place
    for (int64_t i0 = lo; i0 < hi; i0 += 32) {
      const int64_t i = i0 + lane;
      uint32_t d = 0xffffffffu, k = 0u, q = 0u;
      if (i < hi) {
        load(i, k, q);
        d = (k >> shift) & (digits - 1);
      }
      const uint32_t peers = __match_any_sync(0xffffffffu, d);
      if (i < hi) {
        const uint32_t before_me = __popc(peers & ((1u << lane) - 1u));
        const uint32_t at = base[d] + hist[warp * kMaxDigits + d] + before_me;
        key_out[at] = k;
        pos_out[at] = q;
      }
      __syncwarp();
      if (i < hi && lane == __ffs(peers) - 1) hist[warp * kMaxDigits + d] += __popc(peers);
      __syncwarp();
    }
    cluster_sync();  // this pass's keys are in place; every `total` has been read
  }
  // the rows that have a token, and where the ignored tokens begin
  const uint32_t* key = p.key[p.passes & 1];
  for (int64_t i = rank * kSortThreads + tid; i < p.N; i += kSortCtas * kSortThreads) {
    const uint32_t k = __ldcg(key + i);
    if (k >= p.V) continue;
    const uint32_t next = i + 1 < p.N ? __ldcg(key + i + 1) : static_cast<uint32_t>(p.V);
    if (next != k && p.bitmap) atomicOr(p.bitmap + (k >> 5), 1u << (k & 31));
    if (next >= p.V) *p.n_sorted = static_cast<uint32_t>(i + 1);
  }
}

// ---------------------------------------------------------------------- sum
constexpr int kSumThreads = 256;
constexpr int kSumVecs = 2;  // 16-byte vectors of a row per thread
constexpr int kMaxChunk = 64;

struct SumParams {
  const void* dY;
  const uint32_t* key;       // sorted
  const uint32_t* pos;
  const uint32_t* n_sorted;
  const uint32_t* bitmap;    // with dW overwritten
  float* dW;
  float* partial;            // [chunks][2][H]: a run that came in, a run that goes on
  int64_t H, V;
  uint32_t nv;               // 16-byte vectors of dY per row
  int32_t chunk;             // sorted entries per CTA
  int32_t chunks;
  int32_t accumulate;
  float scale;
};

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

// dW row piece: (dW +) scale * sum
__device__ __forceinline__ void finish4(float* dst, float4 v, float scale, bool accumulate) {
  float4* d = reinterpret_cast<float4*>(dst);
  v.x *= scale;
  v.y *= scale;
  v.z *= scale;
  v.w *= scale;
  if (accumulate) {
    const float4 o = *d;
    v.x += o.x;
    v.y += o.y;
    v.z += o.z;
    v.w += o.w;
  }
  *d = v;
}

// Rows that no token has, one warp per row.
__device__ void write_zero_rows(const SumParams& p, int64_t block, int64_t blocks) {
  const int lane = threadIdx.x & 31;
  const int64_t h4 = p.H / 4;
  for (int64_t r = block * (kSumThreads / 32) + (threadIdx.x >> 5); r < p.V;
       r += blocks * (kSumThreads / 32)) {
    if ((__ldg(p.bitmap + (r >> 5)) >> (r & 31)) & 1u) continue;
    float4* row = reinterpret_cast<float4*>(p.dW + r * p.H);
    for (int64_t c = lane; c < h4; c += 32) __stcs(row + c, make_float4(0.f, 0.f, 0.f, 0.f));
  }
}

// Grid: x = chunks (then CTAs that write zero rows), y = slices of the row.
template <int ELT>
__global__ void __launch_bounds__(kSumThreads) embed_sum_kernel(const SumParams p) {
  if (static_cast<int>(blockIdx.x) >= p.chunks) {
    write_zero_rows(p, (blockIdx.x - p.chunks) * gridDim.y + blockIdx.y,
                    static_cast<int64_t>(gridDim.x - p.chunks) * gridDim.y);
    return;
  }
  __shared__ uint32_t s_key[kMaxChunk + 2];  // with the neighbours on both sides
  __shared__ uint32_t s_pos[kMaxChunk];
  const int64_t n = *p.n_sorted;
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * p.chunk;
  if (i0 >= n) return;
  const int cnt = static_cast<int>(n - i0 < p.chunk ? n - i0 : p.chunk);
  constexpr uint32_t kNone = 0xffffffffu;  // no row has this id (ids < 2^31)
  for (int t = threadIdx.x; t < cnt + 2; t += kSumThreads) {
    const int64_t i = i0 + t - 1;
    s_key[t] = (i >= 0 && i < n) ? __ldg(p.key + i) : kNone;
    if (t >= 1 && t <= cnt) s_pos[t - 1] = __ldg(p.pos + i);
  }
  __syncthreads();
  const uint4* dY = static_cast<const uint4*>(p.dY);
  const uint32_t c0 = blockIdx.y * (kSumThreads * kSumVecs) + threadIdx.x;
  Acc<ELT> acc[kSumVecs];
#pragma unroll
  for (int u = 0; u < kSumVecs; ++u) acc[u].zero();
  bool came_in = s_key[0] == s_key[1];
  constexpr int kAhead = 4;  // rows in flight
  for (int j0 = 0; j0 < cnt; j0 += kAhead) {
    uint4 v[kAhead][kSumVecs];
#pragma unroll
    for (int a = 0; a < kAhead; ++a)
#pragma unroll
      for (int u = 0; u < kSumVecs; ++u) {
        const uint32_t c = c0 + u * kSumThreads;
        if (j0 + a < cnt && c < p.nv)
          v[a][u] = __ldcs(dY + static_cast<int64_t>(s_pos[j0 + a]) * p.nv + c);
      }
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int j = j0 + a;
      if (j >= cnt) break;
#pragma unroll
      for (int u = 0; u < kSumVecs; ++u)
        if (c0 + u * kSumThreads < p.nv) acc[u].add(v[a][u]);
      if (s_key[j + 2] == s_key[j + 1] && j + 1 < cnt) continue;  // the run goes on here
      const bool goes_on = s_key[j + 2] == s_key[j + 1];
      constexpr int kN = Acc<ELT>::kN;
#pragma unroll
      for (int u = 0; u < kSumVecs; ++u) {
        const uint32_t c = c0 + u * kSumThreads;
        if (c < p.nv) {
          if (came_in || goes_on) {
            const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (came_in ? 0 : 1);
            acc[u].put(p.partial + slot * p.H + static_cast<int64_t>(c) * kN);
          } else {
            float* dst = p.dW + static_cast<int64_t>(s_key[j + 1]) * p.H +
                         static_cast<int64_t>(c) * kN;
#pragma unroll
            for (int k = 0; k < kN; k += 4)
              finish4(dst + k,
                      make_float4(acc[u].a[k], acc[u].a[k + 1], acc[u].a[k + 2], acc[u].a[k + 3]),
                      p.scale, p.accumulate != 0);
          }
        }
        acc[u].zero();
      }
      came_in = false;
    }
  }
}

// --------------------------------------------------------------------- join
// CTA (c, y): if a run begins in chunk c and goes on into chunk c + 1, adds
// its partial rows: chunk c's second slot, then the first slot of each chunk
// up to the one where the run ends.  Eight groups of threads take contiguous
// shares of those chunks; their sums are added in order.
constexpr int kJoinCols = 32;    // float4 columns per CTA
constexpr int kJoinGroups = 8;
constexpr int kJoinThreads = kJoinCols * kJoinGroups;

__global__ void __launch_bounds__(kJoinThreads) embed_join_kernel(const SumParams p) {
  const int64_t n = *p.n_sorted;
  const int64_t C = p.chunk;
  const int64_t c = blockIdx.x;
  const int64_t after = (c + 1) * C;  // first entry of the next chunk
  if (after >= n) return;
  const uint32_t k = __ldg(p.key + after);
  if (__ldg(p.key + after - 1) != k) return;                        // no run goes on
  if (c > 0 && __ldg(p.key + c * C) == k && __ldg(p.key + c * C - 1) == k) return;  // began earlier
  // chunks c+1 .. last begin with the run's id
  int64_t last = c;
  for (;;) {
    const int64_t e = (last + 1 + threadIdx.x) * C;
    const int hit = __syncthreads_count(e < n && __ldg(p.key + e) == k);
    last += hit;
    if (hit < kJoinThreads) break;
  }
  const int group = threadIdx.x / kJoinCols, col = threadIdx.x % kJoinCols;
  const int64_t h4 = p.H / 4;
  const int64_t x = static_cast<int64_t>(blockIdx.y) * kJoinCols + col;
  const int64_t parts = last - c;  // of the first-slot partials
  const int64_t share = (parts + kJoinGroups - 1) / kJoinGroups;
  const int64_t lo = c + 1 + group * share;
  const int64_t hi = lo + share < last + 1 ? lo + share : last + 1;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  const float4* part = reinterpret_cast<const float4*>(p.partial);
  if (x < h4) {
    if (group == 0) s = __ldcs(part + (2 * c + 1) * h4 + x);
#pragma unroll 8
    for (int64_t q = lo; q < hi; ++q) {
      const float4 v = __ldcs(part + 2 * q * h4 + x);
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
  }
  __shared__ float4 s_part[kJoinGroups][kJoinCols];
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
  if (scale != scale) return host_error(FLCE_ERR_ARG, "%s: scale is NaN", who);
  const int elt = dtype == FLCE_FP32 ? 4 : 2;
  if ((H * elt) % 16 != 0)
    return host_error(FLCE_ERR_ALIGN, "%s: H * sizeof(element) = %lld is not a multiple of 16",
                      who, static_cast<long long>(H * elt));
  if (!aligned16(table) || !aligned16(rows))
    return host_error(FLCE_ERR_ALIGN, "%s: buffers must be 16-byte aligned", who);
  return FLCE_OK;
}

struct BwdPlan {
  int32_t passes, digit_bits, chunk, chunks;
  size_t key[2], pos[2], bitmap, n_sorted, partial, total;
};

// Entries per CTA of the sum: enough CTAs for eight on each of 152 SMs, so
// short inputs spread over the GPU; at most kMaxChunk.
BwdPlan plan_bwd(int64_t N, int64_t H, int64_t V, int elt, bool dense) {
  BwdPlan b{};
  int bits = 1;
  while ((int64_t{1} << bits) <= V) ++bits;  // keys 0 .. V
  b.passes = (bits + kMaxDigitBits - 1) / kMaxDigitBits;
  b.digit_bits = (bits + b.passes - 1) / b.passes;
  const int64_t slices = (H * elt / 16 + kSumThreads * kSumVecs - 1) / (kSumThreads * kSumVecs);
  int64_t c = (N * slices + 152 * 8 - 1) / (152 * 8);
  if (c < 4) c = 4;
  if (c > kMaxChunk) c = kMaxChunk;
  b.chunk = static_cast<int32_t>(c);
  b.chunks = static_cast<int32_t>((N + c - 1) / c);
  size_t o = 0;
  const size_t list = round256(static_cast<size_t>(N) * 4);
  for (int i = 0; i < 2; ++i) {
    b.key[i] = o;
    o += list;
    b.pos[i] = o;
    o += list;
  }
  b.bitmap = o;
  if (dense) o += round256(static_cast<size_t>((V + 31) / 32) * 4);
  b.n_sorted = o;
  o += 256;
  b.partial = o;
  o += round256(static_cast<size_t>(b.chunks) * 2 * static_cast<size_t>(H) * 4);
  b.total = o;
  return b;
}

int run_bwd(const void* dY, const SortParams& sort, const SumParams& sum_in, int elt, int sms,
            cudaStream_t s) {
  SumParams sum = sum_in;
  FLCE_TRY(cudaFuncSetAttribute(embed_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kSortSmem));
  embed_sort_kernel<<<kSortCtas, kSortThreads, kSortSmem, s>>>(sort);
  FLCE_TRY(cudaGetLastError());
  const unsigned slices =
      static_cast<unsigned>((sum.nv + kSumThreads * kSumVecs - 1) / (kSumThreads * kSumVecs));
  unsigned x = static_cast<unsigned>(sum.chunks);
  if (!sum.accumulate) {
    const int64_t want = (sum.V + kSumThreads / 32 - 1) / (kSumThreads / 32);
    const int64_t cap = static_cast<int64_t>(sms) * 8;
    x += static_cast<unsigned>(want < cap ? want : cap);
  }
  if (elt == 2)
    embed_sum_kernel<2><<<dim3(x, slices), kSumThreads, 0, s>>>(sum);
  else
    embed_sum_kernel<4><<<dim3(x, slices), kSumThreads, 0, s>>>(sum);
  FLCE_TRY(cudaGetLastError());
  if (sum.chunks > 1) {
    const unsigned cols = static_cast<unsigned>((sum.H / 4 + kJoinCols - 1) / kJoinCols);
    embed_join_kernel<<<dim3(static_cast<unsigned>(sum.chunks - 1), cols), kJoinThreads, 0, s>>>(
        sum);
    FLCE_TRY(cudaGetLastError());
  }
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
        embed_fwd_kernel<2><<<g, kFwdThreads, 0, call.stream>>>(
            static_cast<const uint4*>(W), id, static_cast<uint4*>(Y), total, nv, V, ignore_index,
            scale, call.status);
      else
        embed_fwd_kernel<4><<<g, kFwdThreads, 0, call.stream>>>(
            static_cast<const uint4*>(W), id, static_cast<uint4*>(Y), total, nv, V, ignore_index,
            scale, call.status);
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
  const BwdPlan b = plan_bwd(N, H, V, elt, accumulate == 0);
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
  for (int i = 0; i < 2; ++i) {
    sp.key[i] = reinterpret_cast<uint32_t*>(w + b.key[i]);
    sp.pos[i] = reinterpret_cast<uint32_t*>(w + b.pos[i]);
  }
  sp.bitmap = accumulate ? nullptr : reinterpret_cast<uint32_t*>(w + b.bitmap);
  sp.n_sorted = reinterpret_cast<uint32_t*>(w + b.n_sorted);
  sp.passes = b.passes;
  sp.digit_bits = b.digit_bits;
  sp.status = call.status;
  SumParams sm{};
  sm.dY = dY;
  sm.key = sp.key[b.passes & 1];
  sm.pos = sp.pos[b.passes & 1];
  sm.n_sorted = sp.n_sorted;
  sm.bitmap = sp.bitmap;
  sm.dW = dW;
  sm.partial = reinterpret_cast<float*>(w + b.partial);
  sm.H = H;
  sm.V = V;
  sm.nv = static_cast<uint32_t>(H * elt / 16);
  sm.chunk = b.chunk;
  sm.chunks = b.chunks;
  sm.accumulate = accumulate != 0 ? 1 : 0;
  sm.scale = scale;
  return call.end(run_bwd(dY, sp, sm, elt, sms, call.stream));
}

}  // extern "C"
