// ckpt_wgrad.cu -- a projection's weight gradient from its input's 8-bit checkpoint:
// dW [O, I] (+)= dY^T X, dY [N, O] bf16, X [N, I] as ckpt.cuh stores it.
//
// X is read back into bf16 scratch, exactly, and multiplied on CTA pairs (tcgen05,
// cta_group::2, tiles of 256 x 256 or 256 x 128, both operands MN-major), as the head's dW is.
// What differs:
//
// Sums.  The tensor core cuts off what falls behind an accumulator's last bit instead of
// rounding it, always towards zero, once for every 16 tokens: 1e-5 of the result after 16384
// of them.  So an accumulator in TMEM takes kPiece k-blocks at most, 2048 tokens, and the pieces
// are added in registers, rounded, in ascending order: eight warps hold a CTA's half of a tile,
// up to 128 sums a thread, and the tensor core goes on with the other accumulator meanwhile.
// (Adding the pieces to dW at L2 took a quarter of the time of the products.)
//   That is a choice of time over digits.  Off from 64-bit sums, by norm, inputs of random sign:
// 6.2e-7 whatever N (7.7e-7 with tokens and channels of different sizes); a plain fp32 product
// 1.4e-7 with 2048 tokens, 3.6e-7 with 8192, 5.7e-7 with 16384.  Inputs of one sign: 2.4e-6, all
// downwards; plain 0.3e-6, 1.0e-6, 1.7e-6.  Pieces of 1024 tokens: 2.8e-7 and 0.9e-6, but 8192 x
// 6144 x 4096 takes 249 us for 242 and 16384 x 512 x 512 32 for 26; of 512: 1.4e-7 and 0.4e-6,
// 293 us.
//
// The last tiles.  Tiles that do not fill a round of all pairs are shared out along the
// tokens, evenly; each pair's share of a tile goes to scratch and a second kernel adds a
// tile's shares in order (8192 x 6144 x 4096: 4 of 384 tiles are left, a sixth round: 260 us
// with it, 235 us shared).  Where that gains less than it costs the last round stays.
//
// Bound by the tensor cores under the board's power limit: 16384 x 14336 x 4096 in 982 us
// when the board is cool (1,960 TFLOP/s), 1,094 to 1,160 back to back (1,660 to 1,760; the measured
// sustained rate of a plain product is 1,715); tensor pipe 96% active.  Small products have 9 to 11 us
// before and behind their tiles, the reading back of X included (2048 x 2048 x 2048: 22 us,
// 1994 x 1000 x 2056: 19).
#include <cmath>

#include "ckpt.cuh"
#include "epilogues.cuh"
#include "host_util.h"
#include "sm103_attn.cuh"

namespace flce {
namespace {

constexpr int kTileM = 2 * BM;          // a pair's tile, TN wide: 256 or 128
constexpr int kPiece = 32;              // k-blocks of 64 tokens in an accumulator
constexpr uint32_t kABytes = BM * 128;  // of A in a stage of one CTA
constexpr int kSumWarps = 8;            // 32 rows of a tile by kSumCols columns each
constexpr int kWgradThreads = 64 + 32 * kSumWarps;

template <int TN>
struct WgradShape {
  static constexpr uint32_t kBBytes = TN / 2 * 128;
  static constexpr int kStages = TN == 256 ? 6 : 8;  // of 32 or 24 KB in each CTA of a pair
  static constexpr int kSumCols = 4 * TN / kSumWarps;
  static constexpr size_t kSmem = 1024 + kStages * (kABytes + kBBytes) +
                                  kSumWarps * STAGING_BUF_BYTES + SMEM_BARRIER_BYTES;
};

// How the tiles are dealt out (GemmGrid for the order of the tiles and k-blocks).
struct WgradPlan {
  GemmGrid g;
  int32_t units;       // pairs
  int32_t whole;       // tiles that one pair does from end to end
  int32_t sharers;     // pairs that share the rest
  int32_t accumulate;
  int32_t tn;          // columns of a tile
  int64_t O, I;
  float* dW;           // of the join
  float* shares;       // [2 sharers][kTileM][tn]
};

// A pair's next work: k-blocks k0 .. k1 of a tile, into dW or into its share `slot`.
struct Item {
  int32_t tile, k0, k1, slot;  // slot < 0: dW
};

// First k-block (of those of all shared tiles, one after the other) of unit u's share.
__host__ __device__ inline int64_t share_start(const WgradPlan& p, int u) {
  const int64_t all = static_cast<int64_t>(p.g.num_m_blk * p.g.num_n_blk - p.whole) * p.g.num_k_blk;
  return u >= p.sharers ? all : all * u / p.sharers;
}

struct Items {
  const WgradPlan& p;
  int unit, tile, segment = 0;
  int64_t at, end;
  __device__ Items(const WgradPlan& plan, int u)
      : p(plan), unit(u), tile(u), at(share_start(plan, u)), end(share_start(plan, u + 1)) {}
  __device__ bool next(Item& it) {
    if (tile < p.whole) {
      it = Item{tile, 0, p.g.num_k_blk, -1};
      tile += p.units;
      return true;
    }
    if (at >= end) return false;
    const int64_t t = at / p.g.num_k_blk;
    it.tile = p.whole + static_cast<int32_t>(t);
    it.k0 = static_cast<int32_t>(at - t * p.g.num_k_blk);
    const int64_t left = end - at;
    it.k1 = it.k0 + left < p.g.num_k_blk ? it.k0 + static_cast<int32_t>(left) : p.g.num_k_blk;
    at += it.k1 - it.k0;
    it.slot = it.k0 == 0 && it.k1 == p.g.num_k_blk ? -1 : 2 * unit + segment;
    ++segment;
    return true;
  }
};

__device__ __forceinline__ int piece_count(const Item& it) {
  return (it.k1 - it.k0 + kPiece - 1) / kPiece;
}
__device__ __forceinline__ int piece_length(const Item& it, int n) {
  return (it.k1 - it.k0 + n - 1) / n;
}

template <int TN>
__global__ void __launch_bounds__(kWgradThreads, 1)
    ckpt_wgrad_kernel(const __grid_constant__ CUtensorMap tmA,
                      const __grid_constant__ CUtensorMap tmB,
                      const __grid_constant__ CUtensorMap tmOut,
                      const __grid_constant__ CUtensorMap tmShares,
                      const __grid_constant__ WgradPlan p) {
  constexpr uint32_t kBox = 128u * 64;  // 64 elements of MN by 64 tokens
  constexpr uint32_t kAdvance = 16u * 128u;
  constexpr uint32_t kIdesc = make_idesc(1, true, true, kTileM, TN);
  using Shape = WgradShape<TN>;
  constexpr int kStages = Shape::kStages, kSumCols = Shape::kSumCols;
  constexpr uint32_t kBBytes = Shape::kBBytes;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* smA = smem;
  uint8_t* smB = smem + kStages * kABytes;
  uint8_t* staging = smB + kStages * kBBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(staging + kSumWarps * STAGING_BUF_BYTES);
  uint64_t* full = bars;                    // [kStages]  (the even CTA's are used)
  uint64_t* empty = bars + kStages;         // [kStages]
  uint64_t* acc_full = bars + 2 * kStages;  // [2]
  uint64_t* acc_empty = acc_full + 2;       // [2]  (the even CTA's are used)
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_base_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_base_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int unit = static_cast<int>(blockIdx.x >> 1);
  int* const status = p.g.status;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], kSumWarps * 2);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmOut);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_base_slot, TMEM_COLS);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the peer's barriers exist before any remote signal
  tc_fence_after();
  const uint32_t tmem_base = *tmem_base_slot;
  // The previous launch writes X and starts only when all before it is done: nothing but the
  // loads of X waits for it.
  if (p.whole < p.g.num_m_blk * p.g.num_n_blk) grid_launch_dependents();  // the join is next

  Items items(p, unit);
  Item it;
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    uint32_t s = 0, round = 0, loads = 0;
    const uint32_t a_base = smem_addr(smA), b_base = smem_addr(smB);
    const uint32_t full_even = mapa_shared(smem_addr(&full[0]), 0);
    bool ok = true, first = true;
    uint32_t early = 0;  // stages whose dY is on its way before X is there
    while (ok && items.next(it)) {
      int mu, n_blk;
      tile_coords(p.g, it.tile, mu, n_blk);
      const int a_mn = uniform(mu * kTileM + static_cast<int>(rank) * BM);
      const int b_mn = uniform(n_blk * TN + static_cast<int>(rank) * (TN / 2));
      auto load_a = [&](uint32_t stage, int kb) {
        if (rank == 0) expect_tx_elected(&full[stage], 2 * (kABytes + kBBytes));
#pragma unroll
        for (int j = 0; j < 2; ++j)
          tma_load_2d_pair_elected(&tmA, full_even + 8 * stage,
                                   a_base + stage * kABytes + j * kBox, a_mn + 64 * j,
                                   kb * 64);
      };
      if (first) {
        first = false;
        for (; early < kStages && it.k0 + static_cast<int>(early) < it.k1; ++early)
          load_a(early, it.k0 + early);
        grid_dependency_wait();
      }
      for (int kb = it.k0; kb < it.k1; ++kb, ++loads) {
        if (loads >= early) {
          if (!uniform_wait(&empty[s], (round & 1) ^ 1, abort_flag, status)) {
            ok = false;
            break;
          }
          load_a(s, kb);
        }
#pragma unroll
        for (int j = 0; j < TN / 128; ++j)
          tma_load_2d_pair_elected(&tmB, full_even + 8 * s, b_base + s * kBBytes + j * kBox,
                                   b_mn + 64 * j, kb * 64);
        if (++s == kStages) {
          s = 0;
          ++round;
        }
      }
    }
    // Every load has landed before this CTA leaves: the even CTA's on its barriers, the
    // odd one's when the MMAs have released them.
    if (lane == 0) {
      const uint32_t n = loads < kStages ? loads : kStages;
      for (uint32_t i = 0; i < n; ++i) {
        const uint32_t q = loads - 1 - i;
        mbar_wait_drain(rank == 0 ? &full[q % kStages] : &empty[q % kStages], (q / kStages) & 1);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ----------------------------------------------------------------- MMA
    if (rank == 0) {
      uint32_t s = 0, round = 0, acc = 0;
      bool ok = true;
      const Operand16 a0(smem_addr(smA), kBox), b0(smem_addr(smB), kBox);
      while (ok && items.next(it)) {
        const int pieces = piece_count(it), length = piece_length(it, pieces);
        for (int k0 = it.k0; ok && k0 < it.k1; k0 += length, ++acc) {
          const uint32_t buf = acc & 1;
          if (!uniform_wait(&acc_empty[buf], ((acc >> 1) & 1) ^ 1, abort_flag, status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d_tmem = tmem_base + buf * TN;
          const int k1 = k0 + length < it.k1 ? k0 + length : it.k1;
          uint32_t add = 0;
          for (int kb = k0; kb < k1; ++kb) {
            if (!uniform_wait(&full[s], round & 1, abort_flag, status)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const Operand16 a = moved(a0, s * kABytes), b = moved(b0, s * kBBytes);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              mma_f16_pair_at(d_tmem, a, k * kAdvance, b, k * kAdvance, kIdesc, add);
              add = 1;
            }
            commit_pair_elected(&empty[s], 0x3);
            if (++s == kStages) {
              s = 0;
              ++round;
            }
          }
          if (ok) commit_pair_elected(&acc_full[buf], 0x3);
        }
      }
      commit_pair_elected(drain, 0x1);
      if (lane == 0) mbar_wait_drain(drain, 0);
      __syncwarp();
    }
  } else {
    // ---------------------------------------------------------------- sums
    const int q = warp & 3;                        // TMEM lanes 32 q .. 32 q + 31
    const int col = ((warp - 2) >> 2) * kSumCols;  // and kSumCols columns from here
    uint8_t* buffer = staging + (warp - 2) * STAGING_BUF_BYTES;
    const uint32_t free_bar = mapa_shared(smem_addr(&acc_empty[0]), 0);
    const uint32_t lanes = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + col;
    uint32_t acc = 0;
    bool ok = true;
    while (ok && items.next(it)) {
      float2 sum[kSumCols / 2];
#pragma unroll
      for (int c = 0; c < kSumCols / 2; ++c) sum[c] = pair(0.f);
      const int length = piece_length(it, piece_count(it));
      for (int k0 = it.k0; k0 < it.k1; k0 += length, ++acc) {
        const uint32_t buf = acc & 1;
        if (!mbar_wait(&acc_full[buf], (acc >> 1) & 1, abort_flag, status)) {
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int u = 0; u < kSumCols / 16; ++u) {
          uint32_t r[16];
          tmem_ld_32x32b_x16(lanes + buf * TN + 16 * u, r);
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < 8; ++c)
            sum[8 * u + c] = plus2(sum[8 * u + c], make_float2(__uint_as_float(r[2 * c]),
                                                               __uint_as_float(r[2 * c + 1])));
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(free_bar + 8 * buf);
      }
      if (!ok) break;
      int mu, n_blk;
      tile_coords(p.g, it.tile, mu, n_blk);
      const bool share = it.slot >= 0;
      // The last tile's results go out through the ring, which is done with: all at once.
      Items behind = items;
      Item none;
      const bool last = !behind.next(none);
      uint8_t* to = last ? smem + (warp - 2) * (kSumCols / 32) * STAGING_BUF_BYTES : buffer;
      const uint32_t next = last ? STAGING_BUF_BYTES : 0;
      const int x = (share ? 0 : n_blk * TN) + col;
      const int y = (share ? it.slot : mu) * kTileM + static_cast<int>(rank) * BM + 32 * q;
#pragma unroll
      for (int u = 0; u < kSumCols / 32; ++u) {
        if (!last) {
          if (lane == 0) bulk_wait_read<0>();  // the store before has read the buffer
          __syncwarp();
        }
#pragma unroll
        for (int ch = 0; ch < 8; ++ch) {
          const float2 v = sum[16 * u + 2 * ch], w = sum[16 * u + 2 * ch + 1];
          staging_put16(to + u * next, lane, ch, __float_as_uint(v.x), __float_as_uint(v.y),
                        __float_as_uint(w.x), __float_as_uint(w.y));
        }
        if (!share && p.accumulate)
          staging_release<true>(&tmOut, to + u * next, lane, x + 32 * u, y);
        else
          staging_release<false>(share ? &tmShares : &tmOut, to + u * next, lane, x + 32 * u,
                                 y);
      }
    }
    if (lane == 0) bulk_wait<0>();  // stores done before shared memory goes away
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA leaves while the pair still uses it
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, TMEM_COLS);
  }
}

// dW of the shared tiles: each the sum of its shares, in ascending order of their tokens.  A
// CTA has kJoinRows rows of a tile, a thread four columns of one, kJoinAtOnce loads in flight.
constexpr int kJoinThreads = 256, kJoinAtOnce = 8;
template <int TN>
constexpr int kJoinRows = kJoinThreads / (TN / 4);

__device__ __forceinline__ void add4(float4& a, const float4& b) {
  a = make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}

template <int TN>
__global__ void __launch_bounds__(kJoinThreads)
    ckpt_wgrad_join_kernel(const __grid_constant__ WgradPlan p) {
  // The units u .. end with some of this tile's k-blocks, and whether unit u ends another tile
  // first: a few long divisions, by one thread.
  __shared__ int found[3];
  const int64_t t = blockIdx.y;  // of the shared tiles
  if (threadIdx.x == 0) {
    const int64_t shared = p.g.num_m_blk * p.g.num_n_blk - p.whole;
    const int64_t k0 = t * p.g.num_k_blk, k1 = k0 + p.g.num_k_blk;
    const int u = static_cast<int>(((k0 + 1) * p.sharers - 1) / (shared * p.g.num_k_blk));
    const int end = static_cast<int>(((t + 1) * p.sharers + shared - 1) / shared);
    const int64_t at = share_start(p, u);
    found[0] = u;
    found[1] = at == k0 && share_start(p, u + 1) >= k1 ? u : end;  // unit u did the whole tile
    found[2] = at < k0;
  }
  __syncthreads();
  const int u = found[0], end = found[1];
  const bool behind = found[2];
  grid_dependency_wait();
  if (end == u) return;
  int mu, n_blk;
  tile_coords(p.g, p.whole + static_cast<int>(t), mu, n_blk);
  const int row = blockIdx.x * kJoinRows<TN> + threadIdx.x / (TN / 4);
  const int quad = threadIdx.x % (TN / 4);
  const int64_t at = mu * static_cast<int64_t>(kTileM) + row;
  if (at >= p.O || n_blk * TN + 4 * quad >= p.I) return;
  const float4* from = reinterpret_cast<const float4*>(p.shares) + row * (TN / 4) + quad;
  constexpr int64_t kSlot = kTileM * TN / 4;
  float4* to = reinterpret_cast<float4*>(p.dW + at * p.I + n_blk * TN + 4 * quad);
  float4 s = p.accumulate ? *to : make_float4(0.f, 0.f, 0.f, 0.f);
  for (int w = u; w < end; w += kJoinAtOnce) {
    float4 a[kJoinAtOnce];
#pragma unroll
    for (int i = 0; i < kJoinAtOnce; ++i)
      a[i] = w + i < end ? from[(2 * (w + i) + (w + i == u && behind ? 1 : 0)) * kSlot]
                         : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kJoinAtOnce; ++i) add4(s, a[i]);
  }
  *to = s;
}

int check(const void* dY, int64_t dY_row, const void* ckpt, int64_t N, int64_t O, int64_t I,
          const float* dW, int32_t dtype) {
  const char* fn = "flce_ckpt_wgrad";
  if (dtype != FLCE_BF16) return host_error(FLCE_ERR_ARG, "%s takes bf16 dY (dtype %d)", fn, dtype);
  const int64_t most = int64_t{1} << 20;
  if (N < 0 || N >= (int64_t{1} << 31) || O < 1 || O > most || I < 1 || I > most)
    return host_error(FLCE_ERR_ARG, "%s: sizes must satisfy 0 <= N < 2^31, 1 <= O, I <= 2^20", fn);
  if (O % 8 != 0 || I % 8 != 0)
    return host_error(FLCE_ERR_ALIGN, "%s: O and I must be multiples of 8", fn);
  if (!dW || (N > 0 && (!dY || !ckpt))) return host_error(FLCE_ERR_ARG, "%s: null pointer", fn);
  if (!aligned16(dW)) return host_error(FLCE_ERR_ALIGN, "%s: dW must be 16-byte aligned", fn);
  if (N == 0) return FLCE_OK;
  if (N > 1 && (dY_row < O || dY_row >= (int64_t{1} << 38)))
    return host_error(FLCE_ERR_ARG, "%s: row stride must be at least O", fn);
  if (!aligned16(dY) || !aligned16(ckpt) || (N > 1 && dY_row % 8 != 0))
    return host_error(FLCE_ERR_ALIGN,
                      "%s: buffers must be 16-byte aligned, dY_row a multiple of 8", fn);
  using wide = __int128;
  const wide w0 = reinterpret_cast<uintptr_t>(dW), w1 = w0 + wide{O} * I * 4;
  const wide y0 = reinterpret_cast<uintptr_t>(dY), c0 = reinterpret_cast<uintptr_t>(ckpt);
  if ((w0 < y0 + ((N - 1) * wide{dY_row} + O) * 2 && y0 < w1) ||
      (w0 < c0 + flce_ckpt_bytes(N, I) && c0 < w1))
    return host_error(FLCE_ERR_ARG, "%s: dW overlaps an input", fn);
  return FLCE_OK;
}

// Boxes of `box` rows by `box` columns of a matrix.
int map_of(CUtensorMap* m, const void* p, CUtensorMapDataType t, int64_t cols, int64_t rows,
           int64_t pitch, uint32_t box, const char* what) {
  const uint64_t dims[2] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(rows)};
  const uint64_t pitches[1] = {static_cast<uint64_t>(pitch)};
  const uint32_t boxes[2] = {box, box};
  return host_tensor_map(m, p, t, 2, dims, pitches, boxes, what);
}

// The tiles of one width dealt out, and an estimate of the time.  A k-block takes a pair 0.34 us
// (0.22 in tiles of 128), a tile's results 5.4 us (2.2) to be written while the next one's
// products run, and there are 11 us (9.5) around the rounds.
//
// The last round's tiles, K k-blocks in all, may be shared by n pairs along the tokens: a share
// takes 0.18 us (0.09) to be written and read, 256 KB (128) each way, the join a launch of
// 4 us.  So they take 0.34 K / n + 0.18 n, least at n = sqrt(0.34 K / 0.18).  One round,
// shared: 20000 x 1000 x 1000 (16 tiles) 168 -> 64 us, 9768 x 184 x 424 (2 tiles) 68 -> 20; the
// last round only, 8192 x 4096 x 4096 (28 of 256 tiles) 178 -> 170.  With 0.06 in place of
// 0.18 65536 x 256 x 256 takes 41 us, not 34.  Where little is expected the pairs keep whole
// tiles, which they read side by side (16384 x 14336 x 4096, 60 of 896 tiles left, back to
// back: 1,148 us, 1,180 with those shared).
WgradPlan deal(int64_t N, int64_t O, int64_t I, int units, int tn, double* us) {
  const double block = tn == 256 ? 0.34 : 0.22, results = tn == 256 ? 5.4 : 2.2;
  const double share = tn == 256 ? 0.18 : 0.09, around = tn == 256 ? 11.0 : 9.5;
  WgradPlan p{};
  p.tn = tn;
  p.g.num_m_blk = static_cast<int32_t>((O + kTileM - 1) / kTileM);
  p.g.num_n_blk = static_cast<int32_t>((I + tn - 1) / tn);
  p.g.num_k_blk = static_cast<int32_t>((N + 63) / 64);
  p.g.raster_n = 1;
  p.g.n_band = 8 * (256 / tn);  // pairs that run together take about 8 x 9 tiles of 256
  p.units = units;
  const int tiles = p.g.num_m_blk * p.g.num_n_blk, left = tiles % units;
  const int rounds = (tiles + units - 1) / units;
  const double tile = block * p.g.num_k_blk, round = tile > results ? tile : results;
  *us = around + (rounds - 1) * round + tile;
  p.whole = tiles;
  p.sharers = 1;
  if (left) {
    int n = static_cast<int>(std::sqrt(left * tile / share));
    n = n < units ? n : units;
    const double shared = n > left ? left * tile / n + share * n + 4.0 : tile;
    if (shared < 0.9 * tile) {
      p.whole = tiles - left;
      p.sharers = n;
      *us += shared - tile;
    }
  }
  if (tiles < units) p.units = p.whole ? tiles : p.sharers;
  return p;
}

// Tiles of 128 columns where they are expected to take less time: where few of 256 leave pairs
// idle (1994 x 1000 x 2056 24.6 -> 18.9 us, 4096 x 2048 x 1024 29.7 -> 23.2), or where there are few
// tokens (52 x 5376 x 992 16.1 -> 11.5).  Where tiles abound those of 256 take
// half as much of L2 (8192 x 4096 x 4096 171 us against 222).
WgradPlan plan(int64_t N, int64_t O, int64_t I, int units, bool accumulate) {
  double wide_us, narrow_us;
  const WgradPlan wide = deal(N, O, I, units, 256, &wide_us);
  const WgradPlan narrow = deal(N, O, I, units, 128, &narrow_us);
  WgradPlan p = narrow_us < 0.95 * wide_us ? narrow : wide;
  p.accumulate = accumulate;
  return p;
}

template <int TN>
cudaError_t launch_products(const CUtensorMap& ma, const CUtensorMap& mb, const CUtensorMap& mw,
                            const CUtensorMap& ms, const WgradPlan& p, cudaStream_t s) {
  static SmemLimit limit;
  const cudaError_t e = limit.raise(ckpt_wgrad_kernel<TN>, WgradShape<TN>::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cfg.gridDim = dim3(static_cast<unsigned>(2 * p.units));
  cfg.blockDim = dim3(kWgradThreads);
  cfg.dynamicSmemBytes = WgradShape<TN>::kSmem;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, ckpt_wgrad_kernel<TN>, ma, mb, mw, ms, p);
}

template <int TN>
cudaError_t launch_join(const WgradPlan& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim =
      dim3(kTileM / kJoinRows<TN>, static_cast<unsigned>(p.g.num_m_blk * p.g.num_n_blk - p.whole));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, ckpt_wgrad_join_kernel<TN>, p);
}

}  // namespace
}  // namespace flce

using namespace flce;

extern "C" int flce_ckpt_wgrad(const void* dY, int64_t dY_row, const void* ckpt, int64_t N,
                               int64_t O, int64_t I, float* dW, int32_t accumulate,
                               const flce_opts* opts) {
  host_clear_error();
  const flce_opts o = opts_or_default(opts);
  int rc = check(dY, dY_row, ckpt, N, O, I, dW, o.dtype);
  if (rc) return rc;
  int sms = 0;
  if ((rc = host_device(&sms))) return rc;
  const WgradPlan all = plan(N, O, I, sms / 2, accumulate != 0);
  const bool shared = N > 0 && all.whole < all.g.num_m_blk * all.g.num_n_blk;
  const size_t x_bytes = round256(static_cast<size_t>(N) * static_cast<size_t>(I) * 2);
  const int64_t share_rows = shared ? 2 * static_cast<int64_t>(all.sharers) * kTileM : 0;
  StepCall call;
  if ((rc = call.begin(o, x_bytes + static_cast<size_t>(share_rows) * all.tn * 4,
                       N > 0 ? StepCall::kKernelClears : StepCall::kCleared)))
    return rc;
  if (N == 0) {
    if (!accumulate) {
      const cudaError_t e =
          cudaMemsetAsync(dW, 0, static_cast<size_t>(O) * static_cast<size_t>(I) * 4, call.stream);
      if (e != cudaSuccess) rc = host_cuda_error(e, "cudaMemsetAsync(dW)");
    }
    return call.end(rc);
  }
  WgradPlan p = all;
  p.g.status = call.status;
  p.O = O;
  p.I = I;
  p.dW = dW;
  p.shares = reinterpret_cast<float*>(call.scratch + x_bytes);
  CUtensorMap ma, mb, mw, ms;
  const auto bf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const auto fp32 = CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
  if ((rc = map_of(&ma, dY, bf16, O, N, (N > 1 ? dY_row : O) * 2, 64, "dY")) ||
      (rc = map_of(&mb, call.scratch, bf16, I, N, I * 2, 64, "X")) ||
      (rc = map_of(&mw, dW, fp32, I, O, I * 4, 32, "dW")))
    return call.end(rc);
  ms = mw;
  if (shared && (rc = map_of(&ms, p.shares, fp32, p.tn, share_rows, p.tn * 4, 32, "shares")))
    return call.end(rc);
  cudaError_t e = launch_ckpt_load(ckpt_view(const_cast<void*>(ckpt), N, I), call.scratch, I, N,
                                   I, 2, call.status, call.stream);
  if (e == cudaSuccess)
    e = p.tn == 256 ? launch_products<256>(ma, mb, mw, ms, p, call.stream)
                    : launch_products<128>(ma, mb, mw, ms, p, call.stream);
  if (e == cudaSuccess && shared)
    e = p.tn == 256 ? launch_join<256>(p, call.stream) : launch_join<128>(p, call.stream);
  if (e != cudaSuccess) rc = host_cuda_error(e, "ckpt_wgrad");
  return call.end(rc);
}
