// attn_fwd.cu -- forward pass of packed causal attention.
//
// A unit of work is 256 query rows (two tiles, A and B) of one query head.
// For each key tile j and each of the two query tiles:
//   MMA      S = Q K_j^T            into TMEM (128 fp32 columns)
//   softmax  one thread per row: running maximum m and sum l,
//            P = 2^(cS - m) as bf16 over S's own columns
//   MMA      O += P V_j             P from TMEM, V_j as it lies in memory
// with c = scale log2(e).  Only the tile on the diagonal is masked, and it is
// a query tile's last one.
//
// One CTA per SM walks the units, deepest first.  Its MMA warp alternates
// between the tiles (PV_A, next S_A, PV_B, next S_B), so the tensor cores work
// on one tile while the other's exponentials are taken, and both tiles share
// one load of K_j and V_j: the operands' way through shared memory (TMA in, MMA
// out) is 256 KB per two tile products at 128 bytes a clock, just what the MMAs
// take.  Measured at 8192 tokens, 32 heads of 128: two CTAs per SM with a tile
// each 210 us; an MMA warp per tile 196 us and this order 171 us, before the
// softmax took its present form (150 us); the MMA warp serving whichever tile is
// ready, so that one may run ahead into the next unit, 172 us (it polls three
// barriers per product).
//
// The maximum that P and O are relative to follows the true one only when it
// has grown by more than 2^8: until then O needs no rescaling, and P <= 2^8,
// l and O stay far inside fp32 and bf16 range.  The quotient O / l does not
// depend on which reference is used.  P is rounded to bf16 (the MMA's operand
// type); l adds the unrounded values.
//
// A key tile may reach past the end of its sequence.  Those columns are
// masked in S; the rows of V there (another sequence's, of any value) are
// cleared in shared memory, since 0 * NaN would reach O.
//
// For the same reason NaN or an infinity in V would reach the rows of its tile that
// do not see it.  A CTA whose outputs are not all finite goes over its units once
// more, carefully: it clears what is not finite in the V tiles on the diagonal and adds
// it, from memory, to the rows that see it (add_nonfinite).  Looking at every such
// tile beforehand took 161 us in place of 149 at the 8192 tokens above (shared memory
// is what the products wait for).  The careful form is a second instance of the same
// code: as a switch at run time it took 152 us, as a function of its own 153.
//
// Roles (320 threads): warps 0-3 softmax and output of tile A, 4-7 of tile B
// (warp w: TMEM lanes 32 (w % 4) ..), warp 8 TMA, warp 9 MMA.
#include <cfloat>

#include "attn.h"
#include "host_util.h"
#include "sm103_attn.cuh"

namespace flce {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr int kTmaWarp = 8, kMmaWarp = 9;
constexpr int kFwdThreads = 10 * 32;
constexpr float kRescale = 8.f;     // log2 of the growth that triggers a rescaling
constexpr uint32_t kTmemCols = 512;

template <int DP>
struct FwdShape {
  static constexpr int kBoxes = DP / 64;
  static constexpr uint32_t kBoxBytes = kTile * 128;             // 128 rows x 64 elements
  static constexpr uint32_t kTileBytes = kBoxes * kBoxBytes;
  static constexpr int kSlots = DP == 128 ? 4 : 8;               // K and V tiles in flight
  static constexpr int kBarriers = 2 * kSlots + 13;              // and a word each of TMEM, abort
  static constexpr uint32_t kStaging = 8 * 4096;                 // one block per softmax warp
  static constexpr uint32_t kSmem =
      (2 + kSlots) * kTileBytes + kStaging + 8 * (kBarriers + 2) + sizeof(AttnTile);
  static_assert(kSmem <= 232448, "shared memory of one CTA");
};

// The units of a CTA: rounds go through the list forwards and backwards in
// turn, so that no CTA always gets the deeper one.
template <bool PLAN>
struct Unit {
  AttnTile t;
  int head;
  int n[2];  // key tiles of the two query tiles (n[1] = 0: one tile only)
  __device__ __forceinline__ bool get(const AttnParams& p, const AttnTile* own, int round,
                                      int total) {
    const int g = static_cast<int>(gridDim.x);
    const int b = static_cast<int>(blockIdx.x);
    const int64_t u = static_cast<int64_t>(round) * g + (round & 1 ? g - 1 - b : b);
    if (u >= total) return false;
    const int i = static_cast<int>(u / p.Hq);
    t = PLAN ? p.tiles[i] : *own;  // without a plan: round 0 only
    head = static_cast<int>(u - static_cast<int64_t>(i) * p.Hq);
    const int nt = (t.len + kTile - 1) / kTile;
    n[0] = 2 * t.tile + 1;
    n[1] = n[0] < nt ? n[0] + 1 : 0;
    return true;
  }
  __device__ __forceinline__ bool get_uniform(const AttnParams& p, const AttnTile* own, int round,
                                              int total) {
    if (!get(p, own, round, total)) return false;
    t.start = uniform(t.start);
    t.tile = uniform(t.tile);
    n[0] = uniform(n[0]);
    n[1] = uniform(n[1]);
    return true;
  }
  __device__ __forceinline__ int depth() const { return n[1] ? n[1] : n[0]; }
};

// Without a plan: this CTA's unit, found from the offsets by a prefix sum over the
// sequences, and its share of the tokens outside them.  Returns the number of
// units of one head.  `sums`: a word per warp.
__device__ int own_unit(const AttnParams& p, AttnTile* own, int32_t* sums) {
  const int b = threadIdx.x, lane = b & 31, warp = b >> 5;
  const int c0 = b < p.B ? p.cu[b] : 0, c1 = b < p.B ? p.cu[b + 1] : 0;
  const bool ok = __syncthreads_or(c0 < 0 || c1 < c0 || c1 > p.T) == 0;
  if (!ok && b == 0 && blockIdx.x == 0 && p.status) atomicOr(p.status, FLCE_DEV_SEQLENS);
  const int unit = kTile * p.unit;
  const int n = ok ? (c1 - c0 + unit - 1) / unit : 0;
  int inc = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) sums[warp] = inc;
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < kFwdThreads / 32; ++w) {
    if (w < warp) before += sums[w];
    all += sums[w];
  }
  const int at = static_cast<int>(blockIdx.x) / p.Hq - (before + inc - n);
  if (at >= 0 && at < n) *own = AttnTile{c0, c1 - c0, at, 0};
  blank_outside<false>(p, ok, static_cast<int64_t>(blockIdx.x) * kFwdThreads + b,
                       static_cast<int64_t>(gridDim.x) * kFwdThreads);
  __syncthreads();
  return all;
}

// Clears rows [valid, 128) of a V tile, and what is not finite in the rows before;
// whether this thread cleared any of the latter.  128 threads, `i` of this one.
template <int BOXES>
__device__ __forceinline__ bool clear_masked_v(uint8_t* tile, int i, int valid) {
  bool found = false;
#pragma unroll 1
  for (int k = 0; k < 8 * BOXES; ++k) {
    const int piece = i + k * kTile, row = (piece >> 3) & (kTile - 1);
    if (row < valid)
      found |= clear_nonfinite_piece(tile + piece * 16);
    else
      st_shared_v4(smem_addr(tile) + piece * 16, 0, 0, 0, 0);
  }
  fence_proxy_async_smem();
  return found;
}

// Where the outcome of a wait goes that no caller asked for (a test for NULL in every
// wait cost the passes with a plan 1.5%).
__device__ int32_t g_unasked;

// The shared memory of a CTA, and its barriers.
template <int DP>
struct FwdShared {
  using S = FwdShape<DP>;
  uint8_t *q, *kv, *staging;   // [2], [kSlots], a block per softmax warp
  uint64_t *kv_full, *kv_empty;         // [kSlots]
  uint64_t *q_full, *q_empty, *drain;
  uint64_t *s_full, *o_full, *o_empty;  // [2], per query tile
  uint64_t* p_full;                     // [2][2]
  uint32_t* tmem_slot;
  volatile int* abort_flag;
  AttnTile* own;
  volatile int* again;  // an output is not finite
  int* nonfinite_v;     // one more than the last round in which V was not, on the diagonal

  __device__ __forceinline__ explicit FwdShared(uint8_t* smem) {
    q = smem;
    kv = q + 2 * S::kTileBytes;
    staging = kv + S::kSlots * S::kTileBytes;
    kv_full = reinterpret_cast<uint64_t*>(staging + S::kStaging);
    kv_empty = kv_full + S::kSlots;
    q_full = kv_empty + S::kSlots;
    q_empty = q_full + 1;
    s_full = q_empty + 1;
    p_full = s_full + 2;
    o_full = p_full + 4;
    o_empty = o_full + 2;
    drain = o_empty + 2;
    tmem_slot = reinterpret_cast<uint32_t*>(kv_full + S::kBarriers);
    abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    own = reinterpret_cast<AttnTile*>(tmem_slot + 2);
    again = reinterpret_cast<volatile int*>(own + 1);
    nonfinite_v = reinterpret_cast<int*>(own + 1) + 1;
  }

  __device__ void init_barriers() const {  // one thread
    for (int i = 0; i < S::kSlots; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int x = 0; x < 2; ++x) {
      mbar_init(&s_full[x], 1);
      mbar_init(&p_full[2 * x], 4);
      mbar_init(&p_full[2 * x + 1], 4);
      mbar_init(&o_full[x], 1);
      mbar_init(&o_empty[x], 4);
    }
    mbar_init(drain, 1);
    fence_mbar_init();
  }
};

// All units of this CTA.  PLAN: units come from the plan's list.  CAREFUL: with V's
// values that are not finite taken out of the products (see the top).
template <int DP, bool PLAN, bool CAREFUL>
__device__ __forceinline__ void run_units(const CUtensorMap& tmQ, const CUtensorMap& tmK,
                                          const CUtensorMap& tmV, const AttnParams& p,
                                          const FwdShared<DP>& sh, uint32_t tmem, int total,
                                          int32_t* status) {
  using S = FwdShape<DP>;
  constexpr int kSlots = S::kSlots;
  constexpr uint32_t TB = S::kTileBytes;
  uint8_t *const smQ = sh.q, *const smKV = sh.kv, *const staging = sh.staging;
  uint64_t *const kv_full = sh.kv_full, *const kv_empty = sh.kv_empty, *const q_full = sh.q_full,
                  *const q_empty = sh.q_empty, *const s_full = sh.s_full,
                  *const p_full = sh.p_full, *const o_full = sh.o_full,
                  *const o_empty = sh.o_empty, *const drain = sh.drain;
  volatile int* const abort_flag = sh.abort_flag;
  const AttnTile* const own = sh.own;
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  Unit<PLAN> w;

  if (warp >= kTmaWarp) {
    if (warp == kTmaWarp) {
      // ------------------------------------------------------------- TMA
      int g = 0, n_q = 0;
      bool ok = true;
      const uint32_t q_dst = smem_addr(smQ), kv_dst = smem_addr(smKV);
      for (int round = 0; ok && w.get_uniform(p, own, round, total); ++round) {
        const int kvh = uniform(w.head / (p.Hq / p.Hkv));
        if (!uniform_wait(q_empty, (round & 1) ^ 1, abort_flag, status)) break;
        const int tiles = w.n[1] ? 2 : 1;
        expect_tx_elected(q_full, tiles * TB);
        for (int x = 0; x < tiles; ++x)
#pragma unroll
          for (int b = 0; b < S::kBoxes; ++b)
            tma_load_3d_elected(&tmQ, q_full, q_dst + x * TB + b * S::kBoxBytes, 64 * b, w.head,
                                w.t.start + (2 * w.t.tile + x) * kTile);
        ++n_q;
        // the next unit's queries on their way into L2: they are loaded only
        // when this unit's last scores are complete
        Unit<PLAN> next;
        if (next.get_uniform(p, own, round + 1, total))
          for (int x = 0; x < (next.n[1] ? 2 : 1); ++x)
#pragma unroll
            for (int b = 0; b < S::kBoxes; ++b)
              tma_prefetch_3d_elected(&tmQ, 64 * b, next.head,
                                      next.t.start + (2 * next.t.tile + x) * kTile);
        const int depth = w.depth();
        for (int j = 0; ok && j < depth; ++j) {
#pragma unroll
          for (int v = 0; v < 2; ++v) {  // K_j, then V_j
            const int s = g % kSlots;
            ok = ok && uniform_wait(&kv_empty[s], ((g / kSlots) & 1) ^ 1, abort_flag, status);
            if (ok) {
              expect_tx_elected(&kv_full[s], TB);
#pragma unroll
              for (int b = 0; b < S::kBoxes; ++b)
                tma_load_3d_elected(v ? &tmV : &tmK, &kv_full[s],
                                    kv_dst + s * TB + b * S::kBoxBytes, 64 * b, kvh,
                                    w.t.start + j * kTile);
              ++g;
            }
          }
        }
      }
      // every load has landed before this CTA's shared memory goes away
      if (lane == 0) {
        if (n_q > 0) mbar_wait_drain(q_full, (n_q - 1) & 1);
        for (int i = g > kSlots ? g - kSlots : 0; i < g; ++i)
          mbar_wait_drain(&kv_full[i % kSlots], (i / kSlots) & 1);
      }
    }
    if (warp == kMmaWarp) {
      // ------------------------------------------------------------- MMA
      constexpr uint32_t kIdescS = make_idesc(1, false, false, kTile, kTile);
      constexpr uint32_t kIdescO = make_idesc(1, false, true, kTile, DP);
      const Operand16 q_op(smem_addr(smQ), 0), k_op(smem_addr(smKV), 0),
          v_op(smem_addr(smKV), S::kBoxBytes);
      const int k_steps = (p.D + 15) / 16;  // columns past D are zeros
      int g = 0;                            // K and V tiles so far
      int n_p[2] = {0, 0}, n_u[2] = {0, 0}; // products P V, and units, per query tile so far
      auto wait_kv = [&](int i) {
        return uniform_wait(&kv_full[i % kSlots], (i / kSlots) & 1, abort_flag, status);
      };
      auto scores = [&](int x, int i) {
        const Operand16 q = moved(q_op, x * TB), k = moved(k_op, (i % kSlots) * TB);
#pragma unroll
        for (int e = 0; e < DP / 16; ++e) {
          const uint32_t off = (e >> 2) * S::kBoxBytes + (e & 3) * 32;
          if (e < k_steps) mma_f16_at(tmem + x * kTile, q, off, k, off, kIdescS, e > 0);
        }
        commit_elected(&s_full[x]);
      };
      bool ok = true;
      int round = 0;
      for (; ok && w.get_uniform(p, own, round, total); ++round) {
        const int depth = w.depth();
        const int last = w.n[1] ? 1 : 0;  // the query tile that uses each key tile last
        ok = uniform_wait(q_full, round & 1, abort_flag, status) && wait_kv(g);
        if (!ok) break;
        scores(0, g);
        if (last) scores(1, g);
        commit_elected(&kv_empty[g % kSlots]);
        if (depth == 1) commit_elected(q_empty);
        for (int j = 0; ok && j < depth; ++j) {
          const int iv = g + 2 * j + 1, ik = iv + 1;
          bool have_k = false;
          ok = wait_kv(iv);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (!ok || x > last) break;
            if (j < w.n[x]) {
              ok = (j > 0 || uniform_wait(&o_empty[x], (n_u[x] & 1) ^ 1, abort_flag, status)) &&
                   uniform_wait(&p_full[2 * x], n_p[x] & 1, abort_flag, status);
              if (!ok) break;
              const Operand16 v = moved(v_op, (iv % kSlots) * TB);
              auto add_pv = [&](int from) {
                tc_fence_after();
#pragma unroll
                for (int e = from; e < from + kTile / 32; ++e)
                  mma_f16_ts_at(tmem + 2 * kTile + x * DP, tmem + x * kTile + 8 * e, v, e * 2048,
                                kIdescO, (j > 0 || e > 0) ? 1u : 0u);
              };
              add_pv(0);
              if (!(ok = uniform_wait(&p_full[2 * x + 1], n_p[x] & 1, abort_flag, status))) break;
              add_pv(kTile / 32);
              ++n_p[x];
              if (j == 0) ++n_u[x];
              if (j == w.n[x] - 1) commit_elected(&o_full[x]);
            }
            if (x == last) commit_elected(&kv_empty[iv % kSlots]);
            if (j + 1 < w.n[x]) {
              if (!have_k) ok = wait_kv(ik);
              if (!ok) break;
              have_k = true;
              scores(x, ik);
            }
            if (x == last && j + 1 < depth) {
              commit_elected(&kv_empty[ik % kSlots]);
              if (j + 2 == depth) commit_elected(q_empty);
            }
          }
        }
        g += 2 * depth;
      }
      commit_elected(drain);  // all MMAs issued by this warp are done
      if (lane == 0) {
        mbar_wait_drain(drain, 0);
        if (!CAREFUL && ok && round > 0) {  // and have arrived everywhere
          for (int i = g > kSlots ? g - kSlots : 0; i < g; ++i)
            mbar_wait_drain(&kv_empty[i % kSlots], (i / kSlots) & 1);
          mbar_wait_drain(q_empty, (round - 1) & 1);
        }
      }
    }
  } else {
    // ----------------------------------------------------- softmax, output
    const int x = warp >> 2;                                  // query tile
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t tS = tmem + x * kTile + lanes, tO = tmem + 2 * kTile + x * DP + lanes;
    const int row = threadIdx.x & (kTile - 1);
    const float c = p.scale * kLog2e;
    bool ok = true;
    int n_s = 0;  // score tiles so far
    int J = 0;    // key tiles before this unit
    int n_u = 0;  // units of this tile so far
    for (int round = 0; ok && w.get(p, own, round, total); J += w.depth(), ++round) {
      const int n = w.n[x];
      if (n == 0) continue;
      const int q0 = (2 * w.t.tile + x) * kTile;
      const int valid = w.t.len - q0 < kTile ? w.t.len - q0 : kTile;  // rows of this tile
      float m = 0.f, l = 0.f;
      for (int j = 0; j < n; ++j, ++n_s) {
        const bool diag = j == n - 1;
        if (CAREFUL && diag) {
          // The other tile's product with this V, if there is one, comes after this
          // tile's, and so after what is cleared here.
          const int iv = 2 * (J + j) + 1, sv = iv % kSlots;
          if (!uniform_wait(&kv_full[sv], (iv / kSlots) & 1, abort_flag, status)) {
            ok = false;
            break;
          }
          if (clear_masked_v<S::kBoxes>(smKV + sv * TB, row, valid))
            atomicMax(sh.nonfinite_v, round + 1);
        }
        if (!uniform_wait(&s_full[x], n_s & 1, abort_flag, status)) {
          ok = false;
          break;
        }
        tc_fence_after();
        float s[kTile];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          tmem_ld_32x32b_x32(tS + 32 * q, reinterpret_cast<uint32_t(&)[32]>(s[32 * q]));
        tmem_ld_wait();
        if (diag) {
#pragma unroll
          for (int i = 0; i < kTile; ++i) s[i] = i > row ? -INFINITY : s[i];
        }
        // independent chains: few warps per scheduler leave latency to hide
        float mxs[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) mxs[k] = max3(s[k], s[k + 8], s[k + 16]);
#pragma unroll
        for (int i = 24; i < 120; i += 16)
#pragma unroll
          for (int k = 0; k < 8; ++k) mxs[k] = max3(mxs[k], s[i + k], s[i + k + 8]);
#pragma unroll
        for (int k = 0; k < 8; ++k) mxs[k] = fmaxf(mxs[k], s[120 + k]);
        const float mx = c * fmaxf(max3(mxs[0], mxs[1], mxs[2]),
                                   max3(max3(mxs[3], mxs[4], mxs[5]), mxs[6], mxs[7]));
        if (j == 0) {
          m = fmaxf(mx, -FLT_MAX);  // a tile may score nothing but -inf (k of infinities)
        } else if (__any_sync(0xffffffffu, mx > m + kRescale)) {
          // S_j complete means every MMA issued before it is: O is at rest.  Rows that
          // need no rescaling keep m (f = 1), so that no row's bits depend on the
          // others of its warp, which may be another sequence's.
          const float mn = mx > m + kRescale ? mx : m;
          const float f = fast_exp2(m - mn);
          m = mn;
          l *= f;
#pragma unroll 1
          for (int q = 0; q < DP / 16; ++q) {
            uint32_t o[16];
            tmem_ld_32x32b_x16(tO + 16 * q, o);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
            tmem_st_32x32b_x16(tO + 16 * q, o);
          }
        }
        if (diag && valid < kTile && !CAREFUL) {
          const int iv = 2 * (J + j) + 1, sv = iv % kSlots;
          if (!uniform_wait(&kv_full[sv], (iv / kSlots) & 1, abort_flag, status)) {
            ok = false;
            break;
          }
          const int per = (kTile - valid) * 8;
          for (int i = row; i < per * S::kBoxes; i += kTile)
            st_shared_v4(smem_addr(smKV) + sv * TB + (i / per) * S::kBoxBytes + valid * 128 +
                             (i % per) * 16, 0, 0, 0, 0);
          fence_proxy_async_smem();
        }
        // P in two halves: the product with the first runs while the second's
        // exponentials are taken
        const float2 c2 = make_float2(c, c), m2 = make_float2(-m, -m);
        float2 sums[2] = {};
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t pk[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            float2 e = fma2(make_float2(s[64 * q + 2 * i], s[64 * q + 2 * i + 1]), c2, m2);
            e.x = fast_exp2(e.x);
            e.y = fast_exp2(e.y);
            sums[i & 1] = add2(sums[i & 1], e);
            pk[i] = pack_bf16x2(e.x, e.y);
          }
          tmem_st_32x32b_x32(tS + 32 * q, pk);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[2 * x + q]);
        }
        const float2 sum = add2(sums[0], sums[1]);
        l += sum.x + sum.y;
      }
      if (!ok || !uniform_wait(&o_full[x], n_u & 1, abort_flag, status)) break;
      ++n_u;
      tc_fence_after();
      const float inv = 1.f / l;
      uint32_t o[DP / 2];
#pragma unroll
      for (int q = 0; q < DP / 32; ++q) {
        uint32_t r[32];
        tmem_ld_32x32b_x32(tO + 32 * q, r);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i)
          o[16 * q + i] = pack_bf16x2(__uint_as_float(r[2 * i]) * inv,
                                      __uint_as_float(r[2 * i + 1]) * inv);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&o_empty[x]);  // O may be overwritten
      const int64_t tok = static_cast<int64_t>(w.t.start) + q0 + row;
      const bool in = row < valid;
      uint16_t* out = static_cast<uint16_t*>(p.o.p) + (tok - lane) * p.o.token + w.head * p.o.head;
#pragma unroll
      for (int b = 0; b < DP / 64; ++b)
        store_rows_bf16(staging + warp * 4096, reinterpret_cast<uint32_t(&)[32]>(o[32 * b]),
                        out + 64 * b, p.o.token, valid - (row - lane), p.D - 64 * b);
      if (in) p.lse[static_cast<int64_t>(w.head) * p.T + tok] = (m + fast_log2(l)) * kLn2;
      if (!CAREFUL) {
        uint32_t any[4] = {};
#pragma unroll
        for (int i = 0; i < DP / 2; ++i) nonfinite_word(o[i], any[i & 3]);
        if (in && nonfinite_found(any)) *sh.again = 1;
      } else if (*reinterpret_cast<volatile int*>(sh.nonfinite_v) > round) {
        // (a later round's mark is at worst a needless look; tile B also lacks what was
        // cleared for tile A)
        const int64_t t0 = static_cast<int64_t>(w.t.start) + 2 * w.t.tile * kTile;
        if (in)
          add_nonfinite(static_cast<const uint16_t*>(p.v.p) + t0 * p.v.token +
                            w.head / (p.Hq / p.Hkv) * p.v.head,
                        p.v.token, static_cast<int>(tok - t0) + 1,
                        static_cast<uint16_t*>(p.o.p) + tok * p.o.token + w.head * p.o.head, 0,
                        p.D, 1.f);
        __syncwarp();
      }
    }
    tc_fence_before();
  }
}

template <int DP, bool PLAN>
__global__ void __launch_bounds__(kFwdThreads, 1)
    attn_fwd_kernel(const __grid_constant__ CUtensorMap tmQ,
                    const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const AttnParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const FwdShared<DP> sh(smem);
  const int warp = uniform(threadIdx.x >> 5);
  if (threadIdx.x == 0) {
    *sh.abort_flag = 0;
    *sh.again = *sh.nonfinite_v = 0;
    sh.init_barriers();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(sh.tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(*sh.tmem_slot);  // S_A, S_B, O_A, O_B
  int32_t* const status = PLAN || p.status ? p.status : &g_unasked;
  int units;
  if (PLAN) {
    grid_dependency_wait();          // the tile list
    units = *p.n_tiles;
  } else {
    units = own_unit(p, sh.own, reinterpret_cast<int32_t*>(sh.staging));
  }
  const int total = uniform(units) * p.Hq;
  run_units<DP, PLAN, false>(tmQ, tmK, tmV, p, sh, tmem, total, status);
  __syncthreads();
  if (*sh.again && !*sh.abort_flag) {  // the same in every thread
    // nothing is in flight: the barriers start afresh
    if (threadIdx.x == 0) {
      for (uint64_t* b = sh.kv_full; b <= sh.drain; ++b) mbar_inval(b);
      sh.init_barriers();
    }
    __syncthreads();
    tc_fence_after();
    run_units<DP, PLAN, true>(tmQ, tmK, tmV, p, sh, tmem, total, status);
    __syncthreads();
  }
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int DP, bool PLAN>
cudaError_t launch_t(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                     const AttnParams& p, int sms, cudaStream_t s) {
  static SmemLimit limit;
  const cudaError_t e = limit.raise(attn_fwd_kernel<DP, PLAN>, FwdShape<DP>::kSmem);
  if (e != cudaSuccess) return e;
  const int64_t most = static_cast<int64_t>(p.max_tiles) * p.Hq;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(static_cast<unsigned>(most < sms ? most : sms));
  cfg.blockDim = dim3(kFwdThreads);
  cfg.dynamicSmemBytes = FwdShape<DP>::kSmem;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = PLAN ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, attn_fwd_kernel<DP, PLAN>, q, k, v, p);
}

}  // namespace

cudaError_t launch_attn_fwd(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                            const AttnParams& p, int sms, cudaStream_t s) {
  if (p.tiles)
    return p.D <= 64 ? launch_t<64, true>(q, k, v, p, sms, s)
                     : launch_t<128, true>(q, k, v, p, sms, s);
  return p.D <= 64 ? launch_t<64, false>(q, k, v, p, sms, s)
                   : launch_t<128, false>(q, k, v, p, sms, s);
}

}  // namespace flce
