// attn_fwd.cu -- forward pass of packed causal attention.
//
// One CTA per (query tile of 128 rows, query head); two CTAs per SM, so that
// one CTA's MMAs run while the other's exponentials do.  For each key tile j:
//   MMA      S = Q K_j^T            into TMEM (128 fp32 columns)
//   softmax  one thread per row: running maximum m and sum l, P = 2^(cS - m)
//            as bf16 over S's own columns
//   MMA      O += P V_j             P from TMEM, V_j as it lies in memory
// with c = scale log2(e).  Only the tile on the diagonal is masked, and it is
// the last one.
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
// Roles (192 threads): warps 0-3 softmax and output, warp 4 TMA, warp 5 MMA.
#include "attn.h"
#include "host_util.h"
#include "sm103_attn.cuh"

namespace flce {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr int kFwdThreads = 192;
constexpr float kRescale = 8.f;  // log2 of the growth that triggers a rescaling

template <int DP>
struct FwdShape {
  static constexpr int kBoxes = DP / 64;
  static constexpr uint32_t kBoxBytes = kTile * 128;             // 128 rows x 64 elements
  static constexpr uint32_t kTileBytes = kBoxes * kBoxBytes;
  // K and V tiles in flight; with the query tile this leaves room for two
  // CTAs on an SM and no more (TMEM holds two)
  static constexpr int kSlots = DP == 128 ? 2 : 4;
  static constexpr uint32_t kSmem = 1024 + (1 + kSlots) * kTileBytes + 256;
};

constexpr uint32_t kTmemCols = 256;  // S (128) and O (DP <= 128)

template <int DP>
__global__ void __launch_bounds__(kFwdThreads, 2)
    attn_fwd_kernel(const __grid_constant__ CUtensorMap tmQ,
                    const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const AttnParams p) {
  using S = FwdShape<DP>;
  constexpr int kSlots = S::kSlots;
  const int h = static_cast<int>(blockIdx.x % p.Hq);
  const int idx = static_cast<int>(blockIdx.x / p.Hq);
  grid_dependency_wait();  // the tile list
  if (idx >= *p.n_tiles) return;
  const AttnTile t = p.tiles[idx];
  const int n_kv = t.tile + 1;
  const int kvh = h / (p.Hq / p.Hkv);

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* smQ = smem;
  uint8_t* smKV = smem + S::kTileBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smKV + kSlots * S::kTileBytes);
  uint64_t* q_full = bars;
  uint64_t* kv_full = bars + 1;               // [kSlots]
  uint64_t* kv_empty = kv_full + kSlots;      // [kSlots]
  uint64_t* s_full = kv_empty + kSlots;
  uint64_t* p_full = s_full + 1;
  uint64_t* o_full = p_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(o_full + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 1);
    }
    mbar_init(s_full, 1);
    mbar_init(p_full, 4);
    mbar_init(o_full, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 5) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tS = *tmem_slot, tO = tS + kTile;
  const int q0 = t.tile * kTile;

  if (warp == 4) {
    // ------------------------------------------------------------- TMA
    if (lane == 0) {
      mbar_arrive_expect_tx(q_full, S::kTileBytes);
#pragma unroll
      for (int b = 0; b < S::kBoxes; ++b)
        tma_load_3d(&tmQ, q_full, smQ + b * S::kBoxBytes, 64 * b, h, t.start + q0);
      int g = 0;
      bool ok = true;
      for (int j = 0; ok && j < n_kv; ++j) {
        for (int w = 0; w < 2; ++w, ++g) {  // K_j, then V_j
          const int s = g % kSlots;
          if (!mbar_wait(&kv_empty[s], ((g / kSlots) & 1) ^ 1, abort_flag, p.status)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&kv_full[s], S::kTileBytes);
#pragma unroll
          for (int b = 0; b < S::kBoxes; ++b)
            tma_load_3d(w ? &tmV : &tmK, &kv_full[s], smKV + s * S::kTileBytes + b * S::kBoxBytes,
                        64 * b, kvh, t.start + j * kTile);
        }
      }
      // every load has landed before this CTA's shared memory goes away
      mbar_wait_drain(q_full, 0);
      for (int i = g > kSlots ? g - kSlots : 0; i < g; ++i)
        mbar_wait_drain(&kv_full[i % kSlots], (i / kSlots) & 1);
    }
  } else if (warp == 5) {
    // ------------------------------------------------------------- MMA
    if (lane == 0) {
      constexpr uint32_t kIdescS = make_idesc(1, false, false, kTile, kTile);
      constexpr uint32_t kIdescO = make_idesc(1, false, true, kTile, DP);
      const uint32_t q_addr = smem_addr(smQ), kv_addr = smem_addr(smKV);
      const int k_steps = (p.D + 15) / 16;  // columns past D are zeros
      bool ok = mbar_wait(q_full, 0, abort_flag, p.status);
      for (int j = 0; ok && j < n_kv; ++j) {
        const int gk = 2 * j, gv = gk + 1;
        const int sk = gk % kSlots, sv = gv % kSlots;
        if (!mbar_wait(&kv_full[sk], (gk / kSlots) & 1, abort_flag, p.status)) break;
        tc_fence_after();
        const uint32_t k_addr = kv_addr + sk * S::kTileBytes;
        for (int k = 0; k < k_steps; ++k) {
          const uint32_t off = (k >> 2) * S::kBoxBytes + (k & 3) * 32;
          mma_f16(tS, smem_desc_sw128(q_addr + off, 0, 1024),
                  smem_desc_sw128(k_addr + off, 0, 1024), kIdescS, k > 0);
        }
        mma_commit(&kv_empty[sk]);
        mma_commit(s_full);
        if (!mbar_wait(&kv_full[sv], (gv / kSlots) & 1, abort_flag, p.status)) break;
        if (!mbar_wait(p_full, j & 1, abort_flag, p.status)) break;
        tc_fence_after();
        const uint32_t v_addr = kv_addr + sv * S::kTileBytes;
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k)
          mma_f16_ts(tO, tS + 8 * k, smem_desc_sw128(v_addr + k * 2048, S::kBoxBytes, 1024),
                     kIdescO, (j > 0 || k > 0) ? 1u : 0u);
        mma_commit(&kv_empty[sv]);
      }
      mma_commit(o_full);  // all MMAs issued by this thread are done
      mbar_wait_drain(o_full, 0);
    }
  } else {
    // --------------------------------------------------- softmax, output
    const uint32_t lanes = static_cast<uint32_t>(32 * warp) << 16;
    const int row = 32 * warp + lane;
    const int valid = t.len - q0 < kTile ? t.len - q0 : kTile;  // rows of the query tile
    const float c = p.scale * kLog2e;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = 0; j < n_kv; ++j) {
      if (!warp_wait(s_full, j & 1, abort_flag, p.status)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const bool diag = j == n_kv - 1;
      float s[kTile];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        tmem_ld_32x32b_x32(tS + lanes + 32 * q,
                           reinterpret_cast<uint32_t(&)[32]>(s[32 * q]));
      tmem_ld_wait();
      if (diag) {
#pragma unroll
        for (int i = 0; i < kTile; ++i) s[i] = i > row ? -INFINITY : s[i];
      }
      // independent chains: two warps per scheduler leave latency to hide
      float mxs[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) mxs[i] = s[i];
#pragma unroll
      for (int i = 8; i < kTile; ++i) mxs[i & 7] = fmaxf(mxs[i & 7], s[i]);
      const float mx = c * fmaxf(fmaxf(fmaxf(mxs[0], mxs[1]), fmaxf(mxs[2], mxs[3])),
                                 fmaxf(fmaxf(mxs[4], mxs[5]), fmaxf(mxs[6], mxs[7])));
      if (j == 0) {
        m = mx;
      } else if (__any_sync(0xffffffffu, mx > m + kRescale)) {
        // S_j complete means every MMA issued before it is: O is at rest
        const float mn = fmaxf(m, mx);
        const float f = fast_exp2(m - mn);
        m = mn;
        l *= f;
#pragma unroll 1
        for (int q = 0; q < DP / 32; ++q) {
          uint32_t o[32];
          tmem_ld_32x32b_x32(tO + lanes + 32 * q, o);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
          tmem_st_32x32b_x32(tO + lanes + 32 * q, o);
        }
      }
      float2 sums[4] = {};
      const float2 c2 = make_float2(c, c), m2 = make_float2(-m, -m);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float2 e = fma2(make_float2(s[32 * q + 2 * i], s[32 * q + 2 * i + 1]), c2, m2);
          e.x = fast_exp2(e.x);
          e.y = fast_exp2(e.y);
          sums[i & 3] = add2(sums[i & 3], e);
          pk[i] = pack_bf16x2(e.x, e.y);
        }
        tmem_st_32x32b_x16(tS + lanes + 16 * q, pk);
      }
      const float2 sum = add2(add2(sums[0], sums[1]), add2(sums[2], sums[3]));
      l += sum.x + sum.y;
      tmem_st_wait();
      if (diag && valid < kTile) {
        const int gv = 2 * j + 1, sv = gv % kSlots;
        if (!warp_wait(&kv_full[sv], (gv / kSlots) & 1, abort_flag, p.status)) {
          ok = false;
          break;
        }
        uint8_t* v = smKV + sv * S::kTileBytes;
        for (int i = threadIdx.x; i < (kTile - valid) * 8 * S::kBoxes; i += kTile) {
          const int b = i / ((kTile - valid) * 8), r = i % ((kTile - valid) * 8);
          st_shared_v4(smem_addr(v) + b * S::kBoxBytes + valid * 128 + r * 16, 0, 0, 0, 0);
        }
        fence_proxy_async_smem();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full);
    }
    if (ok && warp_wait(o_full, 0, abort_flag, p.status)) {
      tc_fence_after();
      const float inv = 1.f / l;
      const int64_t tok = static_cast<int64_t>(t.start) + q0 + row;
      uint16_t* out = static_cast<uint16_t*>(p.o.p) + tok * p.o.token + h * p.o.head;
#pragma unroll
      for (int q = 0; q < DP / 32; ++q) {
        uint32_t o[32];
        tmem_ld_32x32b_x32(tO + lanes + 32 * q, o);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            w[k] = pack_bf16x2(__uint_as_float(o[8 * i + 2 * k]) * inv,
                               __uint_as_float(o[8 * i + 2 * k + 1]) * inv);
          const int d = 32 * q + 8 * i;
          if (row < valid && d < p.D)
            *reinterpret_cast<uint4*>(out + d) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      if (row < valid) p.lse[static_cast<int64_t>(h) * p.T + tok] = (m + fast_log2(l)) * kLn2;
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tS, kTmemCols);
  }
}

template <int DP>
cudaError_t launch_t(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                     const AttnParams& p, cudaStream_t s) {
  const cudaError_t e =
      cudaFuncSetAttribute(attn_fwd_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(FwdShape<DP>::kSmem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(static_cast<unsigned>(p.max_tiles) * static_cast<unsigned>(p.Hq));
  cfg.blockDim = dim3(kFwdThreads);
  cfg.dynamicSmemBytes = FwdShape<DP>::kSmem;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_fwd_kernel<DP>, q, k, v, p);
}

}  // namespace

cudaError_t launch_attn_fwd(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                            const AttnParams& p, cudaStream_t s) {
  return p.D <= 64 ? launch_t<64>(q, k, v, p, s) : launch_t<128>(q, k, v, p, s);
}

}  // namespace flce
