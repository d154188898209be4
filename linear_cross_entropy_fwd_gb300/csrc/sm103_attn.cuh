// sm103_attn.cuh -- further inline-PTX wrappers, used by the attention and
// orthogonalisation kernels: 3-D TMA loads, MMAs whose A operand lies in
// TMEM, stores to TMEM, and pairs of fp32 operations.
#pragma once
#include "sm103.cuh"

namespace flce {

// ------------------------------------------- issue by a converged warp
// The MMA and TMA warps run their loops with all 32 lanes and let one elected
// lane issue: what they compute then stays in uniform registers, where these
// instructions take their operands from.  Issued from a branch that one lane
// takes, four 64-clock MMAs with their wait and commit took 565 clocks, by a
// converged warp 367 (eight: 774 and 592).

// The same value in every lane, known to be so.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// mbar_wait that looks at the clock and the abort flag only now and then: most
// waits here end within a few hundred clocks, and reading the clock takes
// about as long.
__device__ __forceinline__ bool mbar_spin(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                          int* status) {
  const uint32_t a = smem_addr(bar);
  uint64_t t0 = 0;
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(a, parity)) return true;
    if ((it & 255) == 0) {
      if (*abort_flag) return false;
      const uint64_t t = global_timer_ns();
      if (t0 == 0) t0 = t;
      if (t - t0 > FLCE_WAIT_LIMIT_NS) {
        *abort_flag = 1;
        atomicOr(status, FLCE_DEV_TIMEOUT);
        return false;
      }
    }
  }
}

// mbar_spin by a converged warp; the same answer in every lane.
__device__ __forceinline__ bool uniform_wait(uint64_t* bar, uint32_t parity,
                                             volatile int* abort_flag, int* status) {
  return __all_sync(0xffffffffu, mbar_spin(bar, parity, abort_flag, status)) != 0;
}

__device__ __forceinline__ void mbar_inval(uint64_t* bar) {
  asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// An operand tile in shared memory, 128-byte swizzle (see smem_desc_sw128);
// offsets within the tile are constants added to the descriptor's lower half.
struct Operand16 {
  uint32_t lo, hi;
  __device__ __forceinline__ Operand16(uint32_t addr, uint32_t lbo_bytes) {
    const uint64_t d = smem_desc_sw128(addr, lbo_bytes, 1024);
    lo = static_cast<uint32_t>(d);
    hi = static_cast<uint32_t>(d >> 32);
  }
};

// An operand moved on by `bytes` (a multiple of 16).
__device__ __forceinline__ Operand16 moved(Operand16 o, uint32_t bytes) {
  o.lo += bytes >> 4;
  return o;
}

// D[tmem] (+)= A * B^T with operands `a_off` and `b_off` bytes into their tiles.
__device__ __forceinline__ void mma_f16_at(uint32_t d_tmem, const Operand16& a, uint32_t a_off,
                                           const Operand16& b, uint32_t b_off, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 da, db;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "mov.b64 da, {%1, %2};\n\t"
      "mov.b64 db, {%3, %4};\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, p;\n\t}" ::"r"(d_tmem),
      "r"(a.lo + (a_off >> 4)), "r"(a.hi), "r"(b.lo + (b_off >> 4)), "r"(b.hi), "r"(idesc),
      "r"(accumulate)
      : "memory");
}

// The same over a CTA pair (issued by the even CTA; see mma_f16_pair).
__device__ __forceinline__ void mma_f16_pair_at(uint32_t d_tmem, const Operand16& a,
                                                uint32_t a_off, const Operand16& b,
                                                uint32_t b_off, uint32_t idesc,
                                                uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 da, db;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "mov.b64 da, {%1, %2};\n\t"
      "mov.b64 db, {%3, %4};\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %5, p;\n\t}" ::"r"(d_tmem),
      "r"(a.lo + (a_off >> 4)), "r"(a.hi), "r"(b.lo + (b_off >> 4)), "r"(b.hi), "r"(idesc),
      "r"(accumulate)
      : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem]^T, 16-bit inputs, fp32 accumulate.  Lane i of
// A holds row i, two K elements per 32-bit column (the lower half first).
__device__ __forceinline__ void mma_f16_ts_at(uint32_t d_tmem, uint32_t a_tmem, const Operand16& b,
                                              uint32_t b_off, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 db;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "mov.b64 db, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b.lo + (b_off >> 4)), "r"(b.hi), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Arrive on `bar` when every tcgen05 op that the elected lane issued is done.
__device__ __forceinline__ void commit_elected(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          smem_addr(bar))
      : "memory");
}

// The same for the MMAs of a CTA pair, on the barrier at this offset in every
// CTA of `cta_mask`.
__device__ __forceinline__ void commit_pair_elected(uint64_t* bar, uint16_t cta_mask) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster"
      ".multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(smem_addr(bar)),
      "h"(cta_mask)
      : "memory");
}

__device__ __forceinline__ void expect_tx_elected(uint64_t* bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(
          smem_addr(bar)),
      "r"(bytes)
      : "memory");
}

// 3D tiled load global -> shared; completion counted in bytes on `bar`.
__device__ __forceinline__ void tma_load_3d_elected(const CUtensorMap* map, uint64_t* bar,
                                                    uint32_t dst, int32_t x, int32_t y,
                                                    int32_t z) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// The same within a CTA pair: the byte count completes on the barrier at a
// cluster address (of either CTA).
__device__ __forceinline__ void tma_load_3d_pair_elected(const CUtensorMap* map,
                                                         uint32_t bar_cluster, uint32_t dst,
                                                         int32_t x, int32_t y, int32_t z) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile"
      ".mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// 32 lanes x 16 consecutive 32-bit columns, TMEM -> registers.
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32"
      " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// 32 lanes x 32 consecutive 32-bit columns, registers -> TMEM.
__device__ __forceinline__ void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0],"
      " {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16,"
      " %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0],"
      " {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}

__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(d)
      : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)),
        "l"(reinterpret_cast<const uint64_t&>(c)));
  return reinterpret_cast<const float2&>(d);
}

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(d)
      : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)));
  return reinterpret_cast<const float2&>(d);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// --------------------------------------- NaN and infinities in bf16 tiles
// A product takes 0 times what a mask leaves out, and 0 times NaN or infinity is
// NaN.  So what is not finite in the rows that a tile on the diagonal masks is
// cleared in shared memory, and added again where it does belong.

// `any` (0 at first) becomes NaN in a half when one of w's is not finite: w * 0.
__device__ __forceinline__ void nonfinite_word(uint32_t w, uint32_t& any) {
  asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(any) : "r"(w), "r"(0u));
}

__device__ __forceinline__ bool nonfinite_found(const uint32_t (&any)[4]) {
  return ((any[0] | any[1] | any[2] | any[3]) & 0x7fff7fffu) != 0;
}

// What of a pair of bf16 values is not finite (zeros in place of the rest).
__device__ __forceinline__ uint32_t nonfinite_halves(uint32_t w) {
  const uint32_t lo = (w & 0x7f80u) == 0x7f80u ? 0xffffu : 0u;
  const uint32_t hi = (w & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u;
  return w & (lo | hi);
}

// Clears what is not finite in 16 bytes of shared memory; whether there was any.
__device__ __forceinline__ bool clear_nonfinite_piece(uint8_t* piece) {
  const uint4 q = *reinterpret_cast<const uint4*>(piece);
  uint32_t w[4] = {q.x, q.y, q.z, q.w}, bad = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t b = nonfinite_halves(w[k]);
    bad |= b;
    w[k] ^= b;
  }
  if (bad) st_shared_v4(smem_addr(piece), w[0], w[1], w[2], w[3]);
  return bad != 0;
}

// sum[e] += what is not finite in columns c + e of n rows of a [T, D] bf16 matrix, from
// `row` on in steps of `pitch`, until all sums are NaN.
__device__ __forceinline__ void sum_nonfinite(const uint16_t* row, int64_t pitch, int n, int c,
                                              float (&sum)[8]) {
#pragma unroll 1
  for (int i = 0; i < n; ++i, row += pitch) {
    const uint4 q = *reinterpret_cast<const uint4*>(row + c);
    const uint32_t w[4] = {nonfinite_halves(q.x), nonfinite_halves(q.y), nonfinite_halves(q.z),
                           nonfinite_halves(q.w)};
    if (!(w[0] | w[1] | w[2] | w[3])) continue;
    bool settled = true;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      sum[2 * k] += __uint_as_float(w[k] << 16);
      sum[2 * k + 1] += __uint_as_float(w[k] & 0xffff0000u);
      settled = settled && isnan(sum[2 * k]) && isnan(sum[2 * k + 1]);
    }
    if (settled) break;
  }
}

// dst[c] += f times what is not finite in column c of n rows from `row` on, for the
// columns [c0, c1) in eights; each lane has its own n and dst.
__device__ __forceinline__ void add_nonfinite(const uint16_t* row, int64_t pitch, int n,
                                              uint16_t* dst, int c0, int c1, float f) {
#pragma unroll 1
  for (int c = c0; c < c1; c += 8) {
    float sum[8] = {};
    sum_nonfinite(row, pitch, n, c, sum);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (sum[e] != 0.f)
        dst[c + e] = static_cast<uint16_t>(
            pack_bf16x2(fmaf(sum[e], f, __uint_as_float(uint32_t{dst[c + e]} << 16)), 0.f));
  }
}

// Fetch a 3D box into L2 ahead of its load.
__device__ __forceinline__ void tma_prefetch_3d_elected(const CUtensorMap* map, int32_t x,
                                                        int32_t y, int32_t z) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];\n\t}" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(x), "r"(y), "r"(z)
      : "memory");
}

// 32 rows (one per lane) x 64 bf16 columns, packed in pairs, to rows `pitch`
// elements apart.  They go through 4 KB of shared memory, so that a store
// instruction writes whole 128-byte lines (four rows): stored by the lanes that
// hold the rows, 128 x 128 values took 3200 clocks.  Rows from `rows` on and
// columns from `cols` on (a multiple of 8) are left out.
__device__ __forceinline__ void store_rows_bf16(uint8_t* buf, const uint32_t (&v)[32],
                                                uint16_t* dst, int64_t pitch, int rows, int cols) {
  const int lane = threadIdx.x & 31;
  const uint32_t base = smem_addr(buf);
#pragma unroll
  for (int c = 0; c < 8; ++c)
    st_shared_v4(base + lane * 128 + ((c ^ (lane & 7)) << 4), v[4 * c], v[4 * c + 1],
                 v[4 * c + 2], v[4 * c + 3]);
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = 4 * i + (lane >> 3), c = lane & 7;
    const uint4 w = *reinterpret_cast<const uint4*>(buf + r * 128 + ((c ^ (r & 7)) << 4));
    if (r < rows && 8 * c < cols) *reinterpret_cast<uint4*>(dst + r * pitch + 8 * c) = w;
  }
  __syncwarp();
}

}  // namespace flce
