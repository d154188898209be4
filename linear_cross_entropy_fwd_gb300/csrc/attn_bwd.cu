// attn_bwd.cu -- gradients of packed causal attention, in two kernels that
// each own their outputs: no atomics, the same bits on every run.
//
//   dkdv  one CTA per (key tile of 128 rows, kv head); for every query head of
//         the group and every query tile i that sees the key tile:
//           S^T = K Q_i^T, dP^T = V dO_i^T
//           P^T = 2^(c S^T - lse2_i), dS^T = P^T o (dP^T - delta_i)
//           dV += P^T dO_i, dK += dS^T Q_i     accumulated in TMEM
//   dq    one CTA per (query tile, query head); for every key tile j:
//           S = Q K_j^T, dP = dO V_j^T, dS = P o (dP - delta), dQ += dS K_j
//
// Seven products where one kernel for all three would do with five, adding dQ
// to memory from every CTA; that would make dQ depend on the order of the
// additions (or need one more pass over fp32 partial sums).
//
// Where the key tiles alone leave SMs idle, the query heads of a group are shared
// out over a cluster of up to eight CTAs; their fp32 sums are added in head
// order through distributed shared memory (2048 tokens in eight sequences, 16
// heads of 64 on 4: 44 -> 29 us).
//
// P and dS are rounded to bf16, the type of the MMA operands; sums are fp32.
// Only tiles on the diagonal and at a sequence's end are masked, by selection,
// and rows past the end of the sequence are cleared in shared memory where
// they are summed over (they belong to another sequence and may hold anything).
// So is what is not finite in the rows that a tile on the diagonal masks (0 times it
// would be NaN); it is added again where it belongs.  Such rows are looked for only when
// there is a sign of one: of Q or dO an lse or delta, of K a score, that is not finite.
//
// Roles (320 threads): warps 0-7 elementwise (warp w: TMEM lanes 32 (w % 4) ..,
// columns 64 (w / 4) .. of a tile), warp 8 TMA, warp 9 MMA.
#include "attn.h"
#include "host_util.h"
#include "sm103_attn.cuh"

namespace flce {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kThreads = 320;
constexpr int kEwThreads = 256;
constexpr int kTmaWarp = 8, kMmaWarp = 9;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kBoxBytes = kTile * 128;  // 128 rows x 64 bf16

template <int DP>
struct BwdShape {
  static constexpr int kBoxes = DP / 64;
  static constexpr uint32_t kTileBytes = kBoxes * kBoxBytes;
  static constexpr uint32_t kPBytes = 2 * kBoxBytes;  // 128 x 128 bf16
  // dkdv: K, V, two Q and two dO tiles, P^T, lse2 and delta twice, barriers
  static constexpr uint32_t kSmemDkDv = 6 * kTileBytes + kPBytes + 2048 + 256;
  // dq: Q, dO, three K and two V tiles, barriers
  static constexpr uint32_t kSmemDq = 7 * kTileBytes + 256;
};

__device__ __forceinline__ void named_barrier(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// The same; whether x holds in any of the threads.
__device__ __forceinline__ bool named_barrier_or(int id, int threads, bool x) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "bar.red.or.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"(id), "r"(threads), "r"(static_cast<uint32_t>(x))
      : "memory");
  return any != 0;
}

template <int BOXES>
__device__ __forceinline__ void load_tile(const CUtensorMap* m, uint64_t* bar, uint8_t* dst,
                                          int head, int token) {
#pragma unroll
  for (int b = 0; b < BOXES; ++b)
    tma_load_3d_elected(m, bar, smem_addr(dst) + b * kBoxBytes, 64 * b, head, token);
}

// D = A B^T over the head dimension, both tiles K-major in shared memory.
template <int DP>
__device__ __forceinline__ void mma_over_d(uint32_t d_tmem, const Operand16& a, const Operand16& b,
                                           int k_steps) {
  constexpr uint32_t kIdesc = make_idesc(1, false, false, kTile, kTile);
#pragma unroll
  for (int k = 0; k < DP / 16; ++k) {
    const uint32_t off = (k >> 2) * kBoxBytes + (k & 3) * 32;
    if (k < k_steps) mma_f16_at(d_tmem, a, off, b, off, kIdesc, k > 0);
  }
}

// D (+)= A B over 128 rows of B, B a [128 rows, DP] tile in shared memory
// (MN-major); A in TMEM.
template <int DP>
__device__ __forceinline__ void mma_over_rows_ts(uint32_t d_tmem, uint32_t a_tmem,
                                                 const Operand16& b, bool add) {
  constexpr uint32_t kIdesc = make_idesc(1, false, true, kTile, DP);
#pragma unroll
  for (int k = 0; k < kTile / 16; ++k)
    mma_f16_ts_at(d_tmem, a_tmem + 8 * k, b, k * 2048, kIdesc, (add || k > 0) ? 1u : 0u);
}

// The same with A a K-major [128, 128] tile in shared memory.
template <int DP>
__device__ __forceinline__ void mma_over_rows_ss(uint32_t d_tmem, const Operand16& a,
                                                 const Operand16& b, bool add) {
  constexpr uint32_t kIdesc = make_idesc(1, false, true, kTile, DP);
#pragma unroll
  for (int k = 0; k < kTile / 16; ++k)
    mma_f16_at(d_tmem, a, (k >> 2) * kBoxBytes + (k & 3) * 32, b, k * 2048, kIdesc,
               (add || k > 0) ? 1u : 0u);
}

// Rows [valid, 128) of a tile become zeros, and if `look` is set so does what is not
// finite in the rows before; whether this thread cleared any of the latter (the
// elementwise threads, each its own pieces).
template <int BOXES>
__device__ __forceinline__ bool clear_masked(uint8_t* tile, int valid, bool look) {
  bool found = false;
#pragma unroll 1
  for (int i = threadIdx.x; i < 8 * kTile * BOXES; i += kEwThreads) {
    if (((i >> 3) & (kTile - 1)) >= valid)
      st_shared_v4(smem_addr(tile) + i * 16, 0, 0, 0, 0);
    else if (look)
      found |= clear_nonfinite_piece(tile + i * 16);
  }
  fence_proxy_async_smem();
  return found;
}

// Accumulator columns [c0, c0 + 64) of this warp's rows, times f, to bf16.
__device__ __forceinline__ void store_cols(uint32_t taddr, float f, uint8_t* buf, uint16_t* dst,
                                           int64_t pitch, int rows, int cols) {
  uint32_t v[32];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    uint32_t r[32];
    tmem_ld_32x32b_x32(taddr + 32 * q, r);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 16; ++i)
      v[16 * q + i] =
          pack_bf16x2(__uint_as_float(r[2 * i]) * f, __uint_as_float(r[2 * i + 1]) * f);
  }
  store_rows_bf16(buf, v, dst, pitch, rows, cols);
}

// Accumulator columns [c0, c0 + 64) of this thread's row, in fp32, to a
// [128, DP] matrix in shared memory whose 16-byte pieces are swizzled by row.
template <int DP>
__device__ __forceinline__ void put_partial(uint32_t taddr, uint8_t* mat, int row, int c0) {
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    uint32_t r[32];
    tmem_ld_32x32b_x32(taddr + 32 * q, r);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int piece = (c0 + 32 * q) / 4 + i;
      st_shared_v4(smem_addr(mat) + row * (DP * 4) + ((piece ^ (row & 7)) << 4), r[4 * i],
                   r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
    }
  }
}

// Accumulator columns [c0, c0 + 64) of this thread's row of dV, plus what is not finite
// in dO of n tokens down from t1 (the tile's last, to its key's own), for each of this
// CTA's heads.
__device__ __forceinline__ void add_nonfinite_dO(const AttnParams& p, uint32_t taddr, int c0,
                                                 int head0, int heads, int t1, int n) {
#pragma unroll 1
  for (int c = 0; c < 64; c += 16) {
    uint32_t r[16];
    tmem_ld_32x32b_x16(taddr + c, r);
    tmem_ld_wait();
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      const int col = c0 + c + 8 * part;
      float sum[8] = {};
      if (col < p.D)
        for (int h = head0; h < head0 + heads; ++h)
          sum_nonfinite(static_cast<const uint16_t*>(p.dO.p) + t1 * p.dO.token + h * p.dO.head,
                        -p.dO.token, n, col, sum);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        r[8 * part + e] = __float_as_uint(__uint_as_float(r[8 * part + e]) + sum[e]);
    }
    __syncwarp();
    tmem_st_32x32b_x16(taddr + c, r);
    tmem_st_wait();
  }
}

__device__ __forceinline__ float4 ld_shared_cluster_f4(uint32_t cluster_addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(cluster_addr)
               : "memory");
  return v;
}

// This CTA's share of dV and dK: the sums of the cluster's partial matrices in
// rank order, eight columns at a time.
template <int DP>
__device__ __forceinline__ void add_partials(const AttnParams& p, const uint8_t* mats, int token0,
                                             int rows, int kvh, int share, int split) {
  constexpr int kItems = 2 * kTile * (DP / 8);
  const int per = (kItems + split - 1) / split;
  const int end = (share + 1) * per < kItems ? (share + 1) * per : kItems;
  for (int i = share * per + static_cast<int>(threadIdx.x); i < end; i += kThreads) {
    const int is_k = i / (kTile * (DP / 8));
    const int row = i / (DP / 8) % kTile, c8 = i % (DP / 8);
    if (row >= rows || 8 * c8 >= p.D) continue;
    const uint32_t at = smem_addr(mats) + is_k * (kTile * DP * 4) + row * (DP * 4);
    float v[8] = {};
    for (int r = 0; r < split; ++r) {
      const uint32_t remote = mapa_shared(at, static_cast<uint32_t>(r));
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 f = ld_shared_cluster_f4(remote + (((2 * c8 + h) ^ (row & 7)) << 4));
        v[4 * h] += f.x;
        v[4 * h + 1] += f.y;
        v[4 * h + 2] += f.z;
        v[4 * h + 3] += f.w;
      }
    }
    const float f = is_k ? p.scale : 1.f;
    const AttnOut& o = is_k ? p.dk : p.dv;
    uint16_t* dst = static_cast<uint16_t*>(o.p) + (static_cast<int64_t>(token0) + row) * o.token +
                    kvh * o.head + 8 * c8;
    *reinterpret_cast<uint4*>(dst) =
        make_uint4(pack_bf16x2(v[0] * f, v[1] * f), pack_bf16x2(v[2] * f, v[3] * f),
                   pack_bf16x2(v[4] * f, v[5] * f), pack_bf16x2(v[6] * f, v[7] * f));
  }
}

// ===================================================================== dkdv
template <int DP>
__global__ void __launch_bounds__(kThreads, 1)
    attn_dkdv_kernel(const __grid_constant__ CUtensorMap tmQ,
                     const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ CUtensorMap tmO, const AttnParams p,
                     const int split) {
  using S = BwdShape<DP>;
  constexpr uint32_t TB = S::kTileBytes;
  const int share = static_cast<int>(blockIdx.x) % split;  // this CTA's rank in its cluster
  const int kvh = static_cast<int>(blockIdx.x) / split % p.Hkv;
  const int idx = static_cast<int>(blockIdx.x) / split / p.Hkv;
  grid_dependency_wait();  // the tile list and delta
  // dq needs nothing of this launch: its CTAs may take the SMs that this one's
  // last CTAs leave idle
  grid_launch_dependents();
  if (idx >= *p.n_tiles) return;
  AttnTile t = p.tiles[idx];
  t.start = uniform(t.start);
  t.len = uniform(t.len);
  const int n_q = uniform(t.tile) + 1;                           // query tiles that see this key tile
  const int kt = (t.len + kTile - 1) / kTile - n_q;     // this key tile
  const int group = p.Hq / p.Hkv;
  const int heads = group / split;                      // of this CTA
  const int head0 = kvh * group + share * heads;
  const int total = n_q * heads;                        // (head, query tile) pairs

  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* smK = smem;
  uint8_t* smV = smK + TB;
  uint8_t* smQ = smV + TB;       // [2]
  uint8_t* smO = smQ + 2 * TB;   // [2] dO
  uint8_t* smP = smO + 2 * TB;
  float* rows = reinterpret_cast<float*>(smP + S::kPBytes);  // [2][lse2 128, delta 128]
  uint64_t* bars = reinterpret_cast<uint64_t*>(rows + 512);
  uint64_t* kv_full = bars;
  uint64_t* q_full = bars + 1;    // [2]
  uint64_t* q_empty = bars + 3;   // [2]
  uint64_t* o_full = bars + 5;    // [2]
  uint64_t* o_empty = bars + 7;   // [2]
  uint64_t* s_full = bars + 9;
  uint64_t* dp_full = bars + 10;
  uint64_t* p_full = bars + 11;
  uint64_t* p_empty = bars + 12;
  uint64_t* ds_full = bars + 13;
  uint64_t* acc_full = bars + 14;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 15);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* cleared_dO = abort_flag + 1;  // something in a tile on the diagonal

  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 15; ++i) mbar_init(&bars[i], (i == 11 || i == 13) ? 8 : 1);
    *abort_flag = *cleared_dO = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tS = uniform(*tmem_slot), tDP = tS + kTile, tDV = tDP + kTile, tDK = tDV + DP;

  if (warp == kTmaWarp) {
    expect_tx_elected(kv_full, 2 * TB);
    load_tile<S::kBoxes>(&tmK, kv_full, smK, kvh, t.start + kt * kTile);
    load_tile<S::kBoxes>(&tmV, kv_full, smV, kvh, t.start + kt * kTile);
    int n = 0;  // loads issued per ring: n of Q, n or n - 1 of dO
    int n_o = 0;
    for (int it = 0; it < total; ++it) {
      const int s = it & 1;
      const uint32_t par = ((it >> 1) & 1) ^ 1;
      const int head = head0 + it / n_q;
      const int tok = t.start + (kt + it % n_q) * kTile;
      if (!uniform_wait(&q_empty[s], par, abort_flag, p.status)) break;
      expect_tx_elected(&q_full[s], TB);
      load_tile<S::kBoxes>(&tmQ, &q_full[s], smQ + s * TB, head, tok);
      ++n;
      if (!uniform_wait(&o_empty[s], par, abort_flag, p.status)) break;
      expect_tx_elected(&o_full[s], TB);
      load_tile<S::kBoxes>(&tmO, &o_full[s], smO + s * TB, head, tok);
      ++n_o;
    }
    // every load has landed before this CTA's shared memory goes away
    if (lane == 0) {
      mbar_wait_drain(kv_full, 0);
      for (int i = n > 2 ? n - 2 : 0; i < n; ++i) mbar_wait_drain(&q_full[i & 1], (i >> 1) & 1);
      for (int i = n_o > 2 ? n_o - 2 : 0; i < n_o; ++i)
        mbar_wait_drain(&o_full[i & 1], (i >> 1) & 1);
    }
  } else if (warp == kMmaWarp) {
    // operands over the head dimension, and (r..) over rows
    const Operand16 aK(smem_addr(smK), 0), aV(smem_addr(smV), 0), aQ(smem_addr(smQ), 0),
        aO(smem_addr(smO), 0), aP(smem_addr(smP), 0);
    const Operand16 rQ(smem_addr(smQ), kBoxBytes), rO(smem_addr(smO), kBoxBytes);
    const int k_steps = (p.D + 15) / 16;  // columns past D are zeros
    bool ok = uniform_wait(kv_full, 0, abort_flag, p.status) &&
              uniform_wait(&q_full[0], 0, abort_flag, p.status);
    if (ok) {
      tc_fence_after();
      mma_over_d<DP>(tS, aK, aQ, k_steps);
      commit_elected(s_full);
      ok = uniform_wait(&o_full[0], 0, abort_flag, p.status);
    }
    if (ok) {
      tc_fence_after();
      mma_over_d<DP>(tDP, aV, aO, k_steps);
      commit_elected(dp_full);
    }
    for (int it = 0; ok && it < total; ++it) {
      const int s = it & 1, s1 = s ^ 1;
      const uint32_t par1 = ((it + 1) >> 1) & 1;
      const bool more = it + 1 < total;
      // P^T is in shared memory, and S^T has been read
      if (!uniform_wait(p_full, it & 1, abort_flag, p.status)) break;
      if (more) {
        if (!uniform_wait(&q_full[s1], par1, abort_flag, p.status)) break;
        tc_fence_after();
        mma_over_d<DP>(tS, aK, moved(aQ, s1 * TB), k_steps);
        commit_elected(s_full);
      }
      tc_fence_after();
      mma_over_rows_ss<DP>(tDV, aP, moved(rO, s * TB), it > 0);
      commit_elected(&o_empty[s]);
      commit_elected(p_empty);
      // dS^T is in TMEM, and dP^T has been read
      if (!uniform_wait(ds_full, it & 1, abort_flag, p.status)) break;
      tc_fence_after();
      mma_over_rows_ts<DP>(tDK, tDP, moved(rQ, s * TB), it > 0);
      commit_elected(&q_empty[s]);
      if (more) {
        if (!uniform_wait(&o_full[s1], par1, abort_flag, p.status)) break;
        tc_fence_after();
        mma_over_d<DP>(tDP, aV, moved(aO, s1 * TB), k_steps);
        commit_elected(dp_full);
      }
    }
    commit_elected(acc_full);  // all MMAs issued by this thread are done
    if (lane == 0) mbar_wait_drain(acc_full, 0);
  } else {
    const int quarter = warp & 3, half = warp >> 2;
    const uint32_t lanes = static_cast<uint32_t>(32 * quarter) << 16;
    const int row = 32 * quarter + lane;  // key row
    const int tid = threadIdx.x;
    const float c = p.scale * kLog2e;
    // thread t stages lse2 (t < 128) or delta of one query row per tile
    auto fetch = [&](int it) {
      const int q = (kt + it % n_q) * kTile + (tid & 127);
      if (it >= total || q >= t.len) return 0.f;
      const int64_t at = static_cast<int64_t>(head0 + it / n_q) * p.T + t.start + q;
      return tid < kTile ? p.lse[at] * kLog2e : p.delta[at];
    };
    float next = fetch(0);
    // After a wait has expired the loop goes on without results, so that every
    // warp still meets the others at the named barriers; later waits then
    // return at once.
    bool ok = true;
    for (int it = 0; it < total; ++it) {
      const int s = it & 1;
      const int qt = kt + it % n_q;
      const int valid = t.len - qt * kTile < kTile ? t.len - qt * kTile : kTile;
      const bool masked = qt == kt || valid < kTile;
      float* lse2 = rows + s * 256;
      lse2[tid] = next;
      const bool look = named_barrier_or(
          1, kEwThreads, qt == kt && (__float_as_uint(next) & 0x7f800000u) == 0x7f800000u);
      next = fetch(it + 1);
      const float* dl = lse2 + kTile + 64 * half;
      const float* ls = lse2 + 64 * half;

      ok = uniform_wait(s_full, it & 1, abort_flag, p.status) && ok;
      tc_fence_after();
      float P[64];
#pragma unroll
      for (int q = 0; q < 2; ++q)
        tmem_ld_32x32b_x32(tS + lanes + 64 * half + 32 * q,
                           reinterpret_cast<uint32_t(&)[32]>(P[32 * q]));
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 64; i += 4) {
        const float4 L = *reinterpret_cast<const float4*>(ls + i);
        P[i] = fast_exp2(fmaf(P[i], c, -L.x));
        P[i + 1] = fast_exp2(fmaf(P[i + 1], c, -L.y));
        P[i + 2] = fast_exp2(fmaf(P[i + 2], c, -L.z));
        P[i + 3] = fast_exp2(fmaf(P[i + 3], c, -L.w));
      }
      // columns [lo, hi) of this thread's half are queries that see this key
      const int lo = (qt == kt ? row : 0) - 64 * half, hi = valid - 64 * half;
      if (masked) {
#pragma unroll
        for (int i = 0; i < 64; ++i) P[i] = (i >= lo && i < hi) ? P[i] : 0.f;
      }
      ok = uniform_wait(p_empty, (it & 1) ^ 1, abort_flag, p.status) && ok;
      const uint32_t prow = smem_addr(smP) + half * kBoxBytes + row * 128;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        st_shared_v4(prow + ((i ^ (row & 7)) << 4), pack_bf16x2(P[8 * i], P[8 * i + 1]),
                     pack_bf16x2(P[8 * i + 2], P[8 * i + 3]),
                     pack_bf16x2(P[8 * i + 4], P[8 * i + 5]),
                     pack_bf16x2(P[8 * i + 6], P[8 * i + 7]));
      if (valid < kTile || look) {
        // S^T of this tile is complete, so Q is only read again by dK, and after dP^T
        // (issued before this iteration's wait for P) dO only by dV
        ok = uniform_wait(&o_full[s], (it >> 1) & 1, abort_flag, p.status) && ok;
        ok = uniform_wait(dp_full, it & 1, abort_flag, p.status) && ok;
        if (clear_masked<S::kBoxes>(smO + s * TB, valid, look)) *cleared_dO = 1;
        clear_masked<S::kBoxes>(smQ + s * TB, valid, look);
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full);

      ok = uniform_wait(dp_full, it & 1, abort_flag, p.status) && ok;
      tc_fence_after();
      float d[64];
#pragma unroll
      for (int q = 0; q < 2; ++q)
        tmem_ld_32x32b_x32(tDP + lanes + 64 * half + 32 * q,
                           reinterpret_cast<uint32_t(&)[32]>(d[32 * q]));
      tmem_ld_wait();
      // dS^T goes over columns that the other half's warp reads
      tc_fence_before();
      named_barrier(2 + quarter, 64);
      tc_fence_after();
      uint32_t w[32];
#pragma unroll
      for (int i = 0; i < 64; i += 4) {
        const float4 L = *reinterpret_cast<const float4*>(dl + i);
        d[i] = P[i] * (d[i] - L.x);
        d[i + 1] = P[i + 1] * (d[i + 1] - L.y);
        d[i + 2] = P[i + 2] * (d[i + 2] - L.z);
        d[i + 3] = P[i + 3] * (d[i + 3] - L.w);
      }
      if (masked) {
#pragma unroll
        for (int i = 0; i < 64; ++i) d[i] = (i >= lo && i < hi) ? d[i] : 0.f;
      }
#pragma unroll
      for (int i = 0; i < 32; ++i) w[i] = pack_bf16x2(d[2 * i], d[2 * i + 1]);
      tmem_st_32x32b_x32(tDP + lanes + 32 * half, w);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(ds_full);
    }
    if (uniform_wait(acc_full, 0, abort_flag, p.status) && ok) {
      tc_fence_after();
      // Every MMA is done, and the tiles in shared memory are not needed any
      // more.  The two warps of a row take the 64-column blocks of dV and dK in
      // turn.
      const int key0 = kt * kTile + 32 * quarter;
      const int64_t tok = static_cast<int64_t>(t.start) + key0;
      if (*cleared_dO && half < DP / 64) {
        const int end = (kt + 1) * kTile < t.len ? (kt + 1) * kTile : t.len;
        add_nonfinite_dO(p, tDV + lanes + 64 * half, 64 * half, head0, heads, t.start + end - 1,
                         end - (kt * kTile + row));
      }
      uint16_t* dv = static_cast<uint16_t*>(p.dv.p) + tok * p.dv.token + kvh * p.dv.head;
      uint16_t* dk = static_cast<uint16_t*>(p.dk.p) + tok * p.dk.token + kvh * p.dk.head;
#pragma unroll 1
      for (int b = half; b < DP / 32; b += 2) {
        const bool is_k = b >= DP / 64;
        const int c0 = 64 * (b % (DP / 64));
        const uint32_t acc = (is_k ? tDK : tDV) + lanes + c0;
        if (split > 1)
          put_partial<DP>(acc, smem + is_k * (kTile * DP * 4), row, c0);
        else
          store_cols(acc, is_k ? p.scale : 1.f, smQ + warp * 4096, (is_k ? dk : dv) + c0,
                     is_k ? p.dk.token : p.dv.token, t.len - key0, p.D - c0);
      }
    }
    tc_fence_before();
  }
  __syncwarp();
  if (split > 1) {
    cluster_sync();  // every CTA's partial sums are in its shared memory
    add_partials<DP>(p, smem, t.start + kt * kTile, t.len - kt * kTile, kvh, share, split);
    cluster_sync();  // no CTA leaves while others read it
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tS, kTmemCols);
  }
}

// ======================================================================= dq
// S has two buffers, so S of the next tile is complete before the elementwise
// work of this one is; dS takes the place of its own S, which frees dP as soon
// as it has been read.
template <int DP>
__global__ void __launch_bounds__(kThreads, 1)
    attn_dq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV,
                   const __grid_constant__ CUtensorMap tmO, const AttnParams p) {
  using S = BwdShape<DP>;
  constexpr uint32_t TB = S::kTileBytes;
  const int h = static_cast<int>(blockIdx.x % p.Hq);
  const int idx = static_cast<int>(blockIdx.x / p.Hq);
  // The launch before (dkdv) started when the tile list and delta were complete,
  // so they are; that launch itself need only be complete when this one is.
  if (idx >= *p.n_tiles) {
    grid_dependency_wait();
    return;
  }
  AttnTile t = p.tiles[idx];
  t.start = uniform(t.start);
  t.tile = uniform(t.tile);
  const int n_kv = t.tile + 1;
  const int kvh = h / (p.Hq / p.Hkv);
  const int q0 = t.tile * kTile;

  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* smQ = smem;
  uint8_t* smO = smQ + TB;
  uint8_t* smK = smO + TB;       // [3]
  uint8_t* smV = smK + 3 * TB;   // [2]
  uint64_t* bars = reinterpret_cast<uint64_t*>(smV + 2 * TB);
  uint64_t* qo_full = bars;
  uint64_t* k_full = bars + 1;    // [3]
  uint64_t* k_empty = bars + 4;   // [3]
  uint64_t* v_full = bars + 7;    // [2]
  uint64_t* v_empty = bars + 9;   // [2]
  uint64_t* sdp_full = bars + 11;
  uint64_t* dp_read = bars + 12;
  uint64_t* ds_full = bars + 13;
  uint64_t* acc_full = bars + 14;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 15);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* cleared_k = abort_flag + 1;  // something in the tile on the diagonal

  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 15; ++i) mbar_init(&bars[i], (i == 12 || i == 13) ? 8 : 1);
    *abort_flag = *cleared_k = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tS = uniform(*tmem_slot), tDP = tS + 2 * kTile, tDQ = tDP + kTile;

  if (warp == kTmaWarp) {
    expect_tx_elected(qo_full, 2 * TB);
    load_tile<S::kBoxes>(&tmQ, qo_full, smQ, h, t.start + q0);
    load_tile<S::kBoxes>(&tmO, qo_full, smO, h, t.start + q0);
    int n_k = 0, n_v = 0;
    for (int j = 0; j < n_kv; ++j) {
      const int sk = j % 3, sv = j & 1;
      const int tok = t.start + j * kTile;
      if (!uniform_wait(&k_empty[sk], ((j / 3) & 1) ^ 1, abort_flag, p.status)) break;
      expect_tx_elected(&k_full[sk], TB);
      load_tile<S::kBoxes>(&tmK, &k_full[sk], smK + sk * TB, kvh, tok);
      ++n_k;
      if (!uniform_wait(&v_empty[sv], ((j >> 1) & 1) ^ 1, abort_flag, p.status)) break;
      expect_tx_elected(&v_full[sv], TB);
      load_tile<S::kBoxes>(&tmV, &v_full[sv], smV + sv * TB, kvh, tok);
      ++n_v;
    }
    if (lane == 0) {
      mbar_wait_drain(qo_full, 0);
      for (int i = n_k > 3 ? n_k - 3 : 0; i < n_k; ++i)
        mbar_wait_drain(&k_full[i % 3], (i / 3) & 1);
      for (int i = n_v > 2 ? n_v - 2 : 0; i < n_v; ++i)
        mbar_wait_drain(&v_full[i & 1], (i >> 1) & 1);
    }
  } else if (warp == kMmaWarp) {
    const Operand16 aQ(smem_addr(smQ), 0), aO(smem_addr(smO), 0), aK(smem_addr(smK), 0),
        aV(smem_addr(smV), 0);
    const Operand16 rK(smem_addr(smK), kBoxBytes);  // over rows
    const int k_steps = (p.D + 15) / 16;
    auto issue_s = [&](int j) {
      if (!uniform_wait(&k_full[j % 3], (j / 3) & 1, abort_flag, p.status)) return false;
      tc_fence_after();
      mma_over_d<DP>(tS + (j & 1) * kTile, aQ, moved(aK, (j % 3) * TB), k_steps);
      return true;
    };
    auto issue_dp = [&](int j) {
      if (!uniform_wait(&v_full[j & 1], (j >> 1) & 1, abort_flag, p.status)) return false;
      tc_fence_after();
      mma_over_d<DP>(tDP, aO, moved(aV, (j & 1) * TB), k_steps);
      commit_elected(&v_empty[j & 1]);
      commit_elected(sdp_full);  // S of this tile was issued earlier
      return true;
    };
    bool ok = uniform_wait(qo_full, 0, abort_flag, p.status) && issue_s(0) && issue_dp(0) &&
              (n_kv < 2 || issue_s(1));
    for (int j = 0; ok && j < n_kv; ++j) {
      if (!uniform_wait(dp_read, j & 1, abort_flag, p.status)) break;
      if (j + 1 < n_kv && !issue_dp(j + 1)) break;
      if (!uniform_wait(ds_full, j & 1, abort_flag, p.status)) break;
      tc_fence_after();
      mma_over_rows_ts<DP>(tDQ, tS + (j & 1) * kTile, moved(rK, (j % 3) * TB), j > 0);
      commit_elected(&k_empty[j % 3]);
      if (j + 2 < n_kv && !issue_s(j + 2)) break;
    }
    commit_elected(acc_full);
    if (lane == 0) mbar_wait_drain(acc_full, 0);
  } else {
    const int quarter = warp & 3, half = warp >> 2;
    const uint32_t lanes = static_cast<uint32_t>(32 * quarter) << 16;
    const int row = 32 * quarter + lane;
    const bool in = q0 + row < t.len;
    const int64_t tok = static_cast<int64_t>(t.start) + q0 + row;
    const float c = p.scale * kLog2e;
    const int64_t at = static_cast<int64_t>(h) * p.T + tok;
    const float lse2 = in ? p.lse[at] * kLog2e : 0.f;
    const float delta = in ? p.delta[at] : 0.f;
    bool ok = true;
    for (int j = 0; j < n_kv; ++j) {
      const bool diag = j == n_kv - 1;
      ok = uniform_wait(sdp_full, j & 1, abort_flag, p.status) && ok;
      tc_fence_after();
      const uint32_t tSj = tS + (j & 1) * kTile;
      float P[64], d[64];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        tmem_ld_32x32b_x32(tSj + lanes + 64 * half + 32 * q,
                           reinterpret_cast<uint32_t(&)[32]>(P[32 * q]));
        tmem_ld_32x32b_x32(tDP + lanes + 64 * half + 32 * q,
                           reinterpret_cast<uint32_t(&)[32]>(d[32 * q]));
      }
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(dp_read);
      named_barrier(2 + quarter, 64);  // the other half has read S too
      tc_fence_after();
#pragma unroll
      for (int i = 0; i < 64; ++i) d[i] = fast_exp2(fmaf(P[i], c, -lse2)) * (d[i] - delta);
      bool look = false;
      if (diag) {
        // a row of K that is not finite has no finite score
        float any[4] = {};
#pragma unroll
        for (int i = 0; i < 64; ++i) any[i & 3] = fmaf(P[i], 0.f, any[i & 3]);
        look = named_barrier_or(1, kEwThreads, !(any[0] + any[1] + (any[2] + any[3]) == 0.f));
#pragma unroll
        for (int i = 0; i < 64; ++i) d[i] = i + 64 * half > row ? 0.f : d[i];
      }
      uint32_t w[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) w[i] = pack_bf16x2(d[2 * i], d[2 * i + 1]);
      tmem_st_32x32b_x32(tSj + lanes + 32 * half, w);
      tmem_st_wait();
      // S of this tile is complete, so K is only read again by dQ
      if (diag && (look || t.len - q0 < kTile) &&
          clear_masked<S::kBoxes>(smK + (j % 3) * TB, t.len - q0, look))
        *cleared_k = 1;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(ds_full);
    }
    if (uniform_wait(acc_full, 0, abort_flag, p.status) && ok) {
      tc_fence_after();
      // every MMA is done: the key tiles' buffers stage the stores
      const int r0 = 32 * quarter;
      uint16_t* dq = static_cast<uint16_t*>(p.dq.p) + (tok - lane) * p.dq.token + h * p.dq.head;
      if (half < DP / 64) {
        store_cols(tDQ + lanes + 64 * half, p.scale, smK + warp * 4096, dq + 64 * half, p.dq.token,
                   t.len - q0 - r0, p.D - 64 * half);
        if (*cleared_k && in)  // K times a dS that is 0, if it is finite: NaN
          add_nonfinite(static_cast<const uint16_t*>(p.k.p) +
                            (static_cast<int64_t>(t.start) + q0) * p.k.token + kvh * p.k.head,
                        p.k.token, row + 1, dq + lane * p.dq.token, 64 * half,
                        p.D < 64 * half + 64 ? p.D : 64 * half + 64, 0.f);
        __syncwarp();
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tS, kTmemCols);
  }
  grid_dependency_wait();
}

template <class KernelT, class... Extra>
cudaError_t launch(KernelT kernel, SmemLimit& limit, uint32_t smem, unsigned blocks,
                   unsigned cluster, cudaStream_t s, const CUtensorMap& q, const CUtensorMap& k,
                   const CUtensorMap& v, const CUtensorMap& dO, const AttnParams& p,
                   Extra... extra) {
  const cudaError_t e = limit.raise(kernel, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, q, k, v, dO, p, extra...);
}

template <int DP>
cudaError_t launch_dkdv(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                        const CUtensorMap& dO, const AttnParams& p, int split, cudaStream_t s) {
  static SmemLimit limit;
  const unsigned c = static_cast<unsigned>(split);
  const unsigned blocks = static_cast<unsigned>(p.max_tiles) * static_cast<unsigned>(p.Hkv) * c;
  return launch(attn_dkdv_kernel<DP>, limit, BwdShape<DP>::kSmemDkDv, blocks, c, s, q, k, v, dO, p,
                split);
}

template <int DP>
cudaError_t launch_dq(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                      const CUtensorMap& dO, const AttnParams& p, cudaStream_t s) {
  static SmemLimit limit;
  const unsigned blocks = static_cast<unsigned>(p.max_tiles) * static_cast<unsigned>(p.Hq);
  return launch(attn_dq_kernel<DP>, limit, BwdShape<DP>::kSmemDq, blocks, 1, s, q, k, v, dO, p);
}

// CTAs per key tile and kv head: the fewest that give every SM one, among the
// divisors of the group up to eight (the cluster size that always fits).  The
// 2048 tokens above: one 44 us, two or four 29.
int split_heads(const AttnParams& p, int sms) {
  const int group = p.Hq / p.Hkv;
  const int64_t ctas = static_cast<int64_t>(p.max_tiles) * p.Hkv;
  int best = 1;
  for (int n = 1; n <= 8 && n <= group; ++n) {
    if (group % n != 0) continue;
    best = n;
    if (ctas * n >= sms) break;
  }
  return best;
}

}  // namespace

cudaError_t launch_attn_dkdv(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                             const CUtensorMap& dO, const AttnParams& p, int sms, cudaStream_t s) {
  const int split = split_heads(p, sms);
  return p.D <= 64 ? launch_dkdv<64>(q, k, v, dO, p, split, s)
                   : launch_dkdv<128>(q, k, v, dO, p, split, s);
}

cudaError_t launch_attn_dq(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                           const CUtensorMap& dO, const AttnParams& p, cudaStream_t s) {
  return p.D <= 64 ? launch_dq<64>(q, k, v, dO, p, s) : launch_dq<128>(q, k, v, dO, p, s);
}

}  // namespace flce
