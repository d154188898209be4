// ortho.cu -- orthogonalising an update by Newton-Schulz products.
//
//   X = G / (|G|_F + eps);  repeat: A = X X^T, B = b A + c A^2, X = a X + B X
//
// on [rows, cols] matrices, a batch at a time.  A matrix with more rows than
// columns is transposed on the way in and out (X^T X takes the place of X X^T,
// and the same polynomial results), so here X is k x n with k <= n.
//
// Numbers.  The products run on the tensor cores in fp16 with fp32 sums, X, A
// and B stored as 4096 times their values: the entries of all three are below
// 16 (their singular values are, see check_polynomial), and fp16 then holds
// them to 2^-11 down to 2^-26.  X itself is kept in fp32 beside its fp16 copy,
// and only B X goes through the rounded copies.  Without that, the rounding
// errors of X in directions where X has (almost) nothing grow by a = 3.4 per
// step with X: a nearly low-rank 512 x 512 matrix came out 3e-2 off, against
// 2e-3 with it (bf16 operands: 2e-1 and 3e-3; the result's own rounding to
// bf16 is 1.7e-3).
//
// A and A^2 are symmetric: tiles below the diagonal are computed, and written
// twice.  That makes the flops of a step k^2 n + k^3 + 2 k^2 n.
//
// Launches: norm, split (fp32 and fp16 X), then three GEMMs per step, in three
// shapes with 32 KB stages of A and B: CTA pairs on 256 x 256 tiles, and for small
// matrices 128 x 128 tiles by single CTAs or by clusters of four that share out K.
// For k <= 256 the second and third product are one launch.  (All steps in one
// cooperative launch with a barrier over the grid was built and took longer: 154 us
// for eight 256 x 1024 matrices, when three launches per step took 112.  Between two
// products the barrier, the fences before it and the first loads after it took 4 to
// 5 us, and the next launch no more.)  What a launch takes beside its products: 1 us
// until the one before counts as complete, 1 us for the first operands, 1 to 3 us
// of epilogue.
#include <cmath>

#include "host_util.h"
#include "sm103_attn.cuh"

#include <cuda_fp16.h>

namespace flce {
namespace {

constexpr float kHold = 4096.f;       // stored value / value
constexpr float kUnhold = 1.f / 4096.f;
constexpr uint32_t kBox = 64 * 128;   // 64 rows x 64 fp16
constexpr int kStagingBytes = 4096;   // one 32 x 32 fp32 block per epilogue warp

// How a launch covers its tiles.
enum Shape {
  kPair,    // a cluster of two CTAs per 256 x 256 tile, persistent
  kSingle,  // one CTA per 128 x 128 tile, persistent
  kSplit    // a cluster of four CTAs per 128 x 128 tile, each a quarter of K
};
constexpr int kSplitCtas = 4;

template <Shape SHAPE>
struct Config {
  static constexpr int kCtas = SHAPE == kPair ? 2 : 1;  // that share a tile's rows
  static constexpr int kCluster = SHAPE == kSplit ? kSplitCtas : kCtas;
  static constexpr int kM = 128 * kCtas, kN = SHAPE == kPair ? 256 : 128;  // tile
  // 16 where a tile's time is its latency (256 x 1024 all told 98.9 -> 96.3 us, 768 x
  // 768 115.8 -> 111.7); with the larger tiles the fifth and sixth stage of the ring are
  // worth more (2048 x 2048 221 us, 237 with 16 warps and five stages)
  static constexpr int kEpiWarps = SHAPE == kSingle ? 16 : 8;
  static constexpr int kParts = kEpiWarps / 4;  // warps that share a row of the tile
  static constexpr int kStages = SHAPE == kSingle ? 5 : 6;
  static constexpr uint32_t kABytes = 128 * 128;  // 128 rows x 64 fp16
  static constexpr uint32_t kStageBytes = 2 * kABytes;  // A and B
  static constexpr uint32_t kSmem =
      1024 + kStages * kStageBytes + kEpiWarps * kStagingBytes + 256;
  static constexpr int kThreads = 64 + 32 * kEpiWarps;  // TMA, MMA, epilogue
  static_assert(kSmem <= 232448, "shared memory of a CTA");
};

enum Mode { kGram, kPoly, kUpdate };

struct OrthoParams {
  int32_t m_blk, n_blk, k_blk;    // tiles of one matrix; K blocks of 64
  int32_t tiles;                  // of one matrix (symmetric: on and below the diagonal)
  int32_t batch;
  int32_t symmetric;
  int32_t rows, cols;             // of the output (k x k or k x n)
  int64_t ld;                     // of the fp16 output, in elements
  int64_t stride;                 // between matrices of the fp16 output
  __half* out;                    // A, B or the next X, times 4096
  const __half* gram;             // kPoly: A (same layout as out)
  float* x;                       // kUpdate: X in fp32, [rows, ldx]
  int64_t ldx, x_stride;
  uint16_t* result;               // last kUpdate: bf16 result (out unused)
  int32_t transposed;             // result is [cols, rows]
  int32_t result_vec;             // result rows are whole 16-byte vectors
  float a, b, c;
  int32_t* status;
};

// Tile t of one matrix.
__device__ __forceinline__ void tile_of(const OrthoParams& p, int t, int& mi, int& ni) {
  if (p.symmetric) {
    int i = static_cast<int>((sqrtf(8.f * static_cast<float>(t) + 1.f) - 1.f) * 0.5f);
    while ((i + 1) * (i + 2) / 2 <= t) ++i;
    while (i * (i + 1) / 2 > t) --i;
    mi = i;
    ni = t - i * (i + 1) / 2;
  } else {
    mi = t % p.m_blk;  // a column of blocks together: they share a slab of X
    ni = t / p.m_blk;
  }
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// 32 rows (one per lane) x 32 columns of 16-bit values, packed in pairs, to
// memory through shared memory, so that each row goes out in whole 16-byte pieces
// next to one another.
__device__ __forceinline__ void store_16(uint8_t* buf, const uint32_t (&v)[16], uint16_t* dst,
                                         int64_t ld, int rows, int cols, bool vec) {
  const int lane = threadIdx.x & 31;
  const uint32_t base = smem_addr(buf);
#pragma unroll
  for (int c = 0; c < 4; ++c)
    st_shared_v4(base + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4), v[4 * c], v[4 * c + 1],
                 v[4 * c + 2], v[4 * c + 3]);
  __syncwarp();
  if (vec) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 8 * i + (lane >> 2), c = lane & 3;
      const uint4 w = *reinterpret_cast<const uint4*>(buf + r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
      if (r < rows && 8 * c < cols) *reinterpret_cast<uint4*>(dst + r * ld + 8 * c) = w;
    }
  } else {
    for (int r = 0; r < rows && r < 32; ++r) {
      const int c = lane >> 3;
      const uint16_t w = *reinterpret_cast<const uint16_t*>(
          buf + r * 64 + ((c ^ ((r >> 1) & 3)) << 4) + (lane & 7) * 2);
      if (lane < cols) dst[r * ld + lane] = w;
    }
  }
  __syncwarp();
}

// Column j of the block becomes row j of dst, 16 bytes at a time if `vec` (with
// the last piece of a row written whole: rows are padded), else by element.
__device__ __forceinline__ void store_16_transposed(uint8_t* buf, const uint32_t (&v)[16],
                                                    uint16_t* dst, int64_t ld, int rows, int cols,
                                                    bool vec) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < 32; ++j)
    reinterpret_cast<uint16_t*>(buf)[j * 32 + lane] =
        static_cast<uint16_t>(j & 1 ? v[j >> 1] >> 16 : v[j >> 1] & 0xffffu);
  __syncwarp();
  if (vec) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = 8 * i + (lane >> 2), c = lane & 3;
      const uint4 w = *reinterpret_cast<const uint4*>(buf + j * 64 + c * 16);
      if (j < cols && 8 * c < rows) *reinterpret_cast<uint4*>(dst + j * ld + 8 * c) = w;
    }
  } else {
    for (int j = 0; j < cols && j < 32; ++j)
      if (lane < rows) dst[j * ld + lane] = reinterpret_cast<const uint16_t*>(buf)[j * 32 + lane];
  }
  __syncwarp();
}

// What the epilogue adds the product to: a block of 32 x 32 values of X (fp32)
// or of A (fp16).  Fetched in whole lines (a load instruction covers 4 or 8
// rows) and turned around in shared memory into one row per lane; fetched by
// the lanes that need the rows, a 256 x 256 tile's took 11 us.
template <int MODE>
struct Addend {
  static constexpr int kVecs = MODE == kUpdate ? 8 : 4;  // 16-byte pieces of a row
  static constexpr int kPer = 32 / kVecs;                // elements of a piece
  static constexpr int kRows = 32 / kVecs;               // rows per load instruction
  uint4 v[kVecs];

  __device__ __forceinline__ void fetch(const OrthoParams& p, int bi, int row0, int c0) {
    if (MODE == kGram) return;
    const int lane = threadIdx.x & 31, c = lane % kVecs;
    const int64_t ld = MODE == kUpdate ? p.ldx : p.ld;
    const uint4* src =
        MODE == kUpdate
            ? reinterpret_cast<const uint4*>(p.x + bi * p.x_stride + row0 * ld + c0) + c
            : reinterpret_cast<const uint4*>(p.gram + bi * p.stride + row0 * ld + c0) + c;
    const bool in = kPer * c < p.cols - c0;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int r = kRows * i + lane / kVecs;
      v[i] = make_uint4(0u, 0u, 0u, 0u);
      if (in && row0 + r < p.rows) v[i] = __ldcg(src + r * ld / kPer);
    }
  }
  // `buf`: 4 KB of this warp's
  __device__ __forceinline__ void to_rows(uint8_t* buf, float (&out)[32]) const {
    if (MODE == kGram) return;
    const int lane = threadIdx.x & 31, c = lane % kVecs;
    constexpr int kRowBytes = 16 * kVecs;
    const uint32_t base = smem_addr(buf);
    auto swizzle = [](int r) { return MODE == kUpdate ? r & 7 : (r >> 1) & 3; };
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int r = kRows * i + lane / kVecs;
      st_shared_v4(base + r * kRowBytes + ((c ^ swizzle(r)) << 4), v[i].x, v[i].y, v[i].z, v[i].w);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const uint4 q = *reinterpret_cast<const uint4*>(buf + lane * kRowBytes +
                                                      ((i ^ swizzle(lane)) << 4));
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (MODE == kUpdate) {
          out[4 * i + k] = __uint_as_float(w[k]);
        } else {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
          out[8 * i + 2 * k] = f.x;
          out[8 * i + 2 * k + 1] = f.y;
        }
      }
    }
    __syncwarp();
  }
};

// The update's block, X and its fp16 copy (or the bf16 result, in whole vectors):
// the product goes through shared memory into the layout that the addend was
// fetched in (lane l: columns 4 (l % 8) .., rows l / 8 + 4 i), which is also the one
// to store in.  Turning the addend into rows and both results back took 2.5 times
// the shared memory accesses, and an update of 2048 x 2048 20.7 us instead of 19.0.
// What is left is bound by L2: 40 MB in and out in the 6.5 us of the epilogue.
__device__ __forceinline__ void finish_in_pieces(const OrthoParams& p, const Addend<kUpdate>& add,
                                                 const float (&acc)[32], int bi, int row0, int c0,
                                                 uint8_t* buf) {
  const int lane = threadIdx.x & 31, c = lane & 7;
  const uint32_t base = smem_addr(buf);
#pragma unroll
  for (int k = 0; k < 8; ++k)
    st_shared_v4(base + lane * 128 + ((k ^ (lane & 7)) << 4), __float_as_uint(acc[4 * k]),
                 __float_as_uint(acc[4 * k + 1]), __float_as_uint(acc[4 * k + 2]),
                 __float_as_uint(acc[4 * k + 3]));
  __syncwarp();
  const bool in = c0 + 4 * c < p.cols;
  const int64_t r0 = row0 + (lane >> 3), at = c0 + 4 * c;
  float* x = p.x + bi * p.x_stride + r0 * p.ldx + at;
  uint16_t* h = p.result ? p.result + static_cast<int64_t>(bi) * p.rows * p.cols + r0 * p.cols + at
                         : reinterpret_cast<uint16_t*>(p.out) + bi * p.stride + r0 * p.ld + at;
  const int64_t h_ld = p.result ? p.cols : p.ld;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = 4 * i + (lane >> 3);
    const float4 s = *reinterpret_cast<const float4*>(buf + r * 128 + ((c ^ (r & 7)) << 4));
    constexpr float kU = kUnhold * kUnhold;
    float4 v;
    v.x = fmaf(s.x, kU, p.a * __uint_as_float(add.v[i].x));
    v.y = fmaf(s.y, kU, p.a * __uint_as_float(add.v[i].y));
    v.z = fmaf(s.z, kU, p.a * __uint_as_float(add.v[i].z));
    v.w = fmaf(s.w, kU, p.a * __uint_as_float(add.v[i].w));
    if (!in || row0 + r >= p.rows) continue;
    uint2 w;
    if (p.result) {
      w = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
    } else {
      *reinterpret_cast<float4*>(x + 4 * i * p.ldx) = v;
      w = make_uint2(pack_half2(v.x * kHold, v.y * kHold), pack_half2(v.z * kHold, v.w * kHold));
    }
    *reinterpret_cast<uint2*>(h + 4 * i * h_ld) = w;
  }
  __syncwarp();
}

template <int MODE>
__device__ __forceinline__ void finish_in_pieces(const OrthoParams&, const Addend<MODE>&,
                                                 const float (&)[32], int, int, int, uint8_t*) {}

// A 32 x 32 block of an accumulator (row row0 + lane, columns c0 ..), turned into
// the launch's result and stored.  `acc` holds 4096^2 times the product.
template <int MODE>
__device__ __forceinline__ void finish_block(const OrthoParams& p, const Addend<MODE>& add,
                                             const float (&acc)[32], int bi, int row0, int c0,
                                             bool mirror, uint8_t* buf) {
  const int rows = p.rows - row0, cols = p.cols - c0;
  if (MODE == kUpdate && !(p.result && (p.transposed || !p.result_vec))) {
    finish_in_pieces(p, add, acc, bi, row0, c0, buf);
    return;
  }
  float v[32];
  add.to_rows(buf, v);
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    if (MODE == kGram)
      v[i] = acc[i] * kUnhold;
    else if (MODE == kPoly)
      v[i] = fmaf(p.c * kUnhold, acc[i], p.b * v[i]);
    else
      v[i] = fmaf(acc[i], kUnhold * kUnhold, p.a * v[i]);
  }
  uint32_t w[16];
  if constexpr (MODE == kUpdate) {
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    uint16_t* res = p.result + static_cast<int64_t>(bi) * p.rows * p.cols;
    if (p.transposed)
      store_16_transposed(buf, w, res + static_cast<int64_t>(c0) * p.rows + row0, p.rows, rows,
                          cols, p.result_vec != 0);
    else
      store_16(buf, w, res + static_cast<int64_t>(row0) * p.cols + c0, p.cols, rows, cols, false);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = pack_half2(v[2 * i], v[2 * i + 1]);
    uint16_t* o = reinterpret_cast<uint16_t*>(p.out) + bi * p.stride;
    store_16(buf, w, o + row0 * p.ld + c0, p.ld, rows, cols, true);
    if (mirror) store_16_transposed(buf, w, o + c0 * p.ld + row0, p.ld, rows, cols, true);
  }
}

// 32 rows of an accumulator, columns [col0, col0 + width), block by block;
// `add` holds the first block's addend, fetched before the accumulator was
// complete, and each later one is fetched while the one before it is stored.
template <int MODE>
__device__ __forceinline__ void epilogue(const OrthoParams& p, Addend<MODE>& add, uint32_t taddr,
                                         int bi, int row0, int col0, int width, bool mirror,
                                         uint8_t* buf) {
  if (row0 >= p.rows) return;
#pragma unroll 1
  for (int u = 0; u < width; u += 32) {
    const int c0 = col0 + u;
    if (c0 >= p.cols) break;
    uint32_t r[32];
    tmem_ld_32x32b_x32(taddr + u, r);
    const Addend<MODE> cur = add;
    if (u + 32 < width) add.fetch(p, bi, row0, c0 + 32);
    tmem_ld_wait();
    finish_block<MODE>(p, cur, reinterpret_cast<const float(&)[32]>(r), bi, row0, c0, mirror, buf);
  }
}

__device__ __forceinline__ void st_cluster_v4(uint32_t cluster_addr, uint32_t a, uint32_t b,
                                              uint32_t c, uint32_t d) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(cluster_addr), "r"(a),
               "r"(b), "r"(c), "r"(d)
               : "memory");
}

// This warp's 32 rows and 64 columns of a partial sum, to the CTAs that finish
// them: CTA b of the cluster gets columns [32 b, 32 b + 32) of the tile from each
// CTA's `from`, as a [128, 32] matrix whose 16-byte pieces are swizzled by row.
__device__ __forceinline__ void send_partial(uint32_t taddr, uint8_t* ring, uint32_t from, int row,
                                             int half) {
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    uint32_t r[32];
    tmem_ld_32x32b_x32(taddr + 32 * u, r);
    tmem_ld_wait();
    const uint32_t at = mapa_shared(smem_addr(ring) + from * 16384 + row * 128,
                                    static_cast<uint32_t>(2 * half + u));
#pragma unroll
    for (int i = 0; i < 8; ++i)
      st_cluster_v4(at + ((i ^ (row & 7)) << 4), r[4 * i], r[4 * i + 1], r[4 * i + 2],
                    r[4 * i + 3]);
  }
}

// The sum of the four partial sums that have arrived, in rank order.
__device__ __forceinline__ void sum_partials(const uint8_t* ring, int row, float (&acc)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) acc[i] = 0.f;
#pragma unroll
  for (int from = 0; from < kSplitCtas; ++from)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4 f = *reinterpret_cast<const float4*>(ring + from * 16384 + row * 128 +
                                                        ((i ^ (row & 7)) << 4));
      acc[4 * i] += f.x;
      acc[4 * i + 1] += f.y;
      acc[4 * i + 2] += f.z;
      acc[4 * i + 3] += f.w;
    }
}

// D = A B^T (B K-major) or A B (B_MN: B stored [K, N]), one tile per
// accumulator; the epilogue of a tile runs beside the MMAs of the next.  Both
// operands come from the previous launch.
template <int MODE, Shape SHAPE>
__global__ void __launch_bounds__(Config<SHAPE>::kThreads, 1)
    ortho_gemm(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
               const OrthoParams p) {
  using C = Config<SHAPE>;
  constexpr bool PAIR = C::kCtas == 2, SPLIT = SHAPE == kSplit;
  constexpr bool B_MN = MODE == kUpdate;
  constexpr int kCtas = C::kCtas, kN = C::kN, kStages = C::kStages, kParts = C::kParts;
  constexpr uint32_t kStageBytes = C::kStageBytes;
  constexpr uint32_t kCols = 2 * kN;  // two accumulators
  constexpr uint32_t kIdesc = make_idesc(0, false, B_MN, C::kM, kN);

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* staging = smem + kStages * kStageBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(staging + C::kEpiWarps * kStagingBytes);
  uint64_t* full = bars;                  // [kStages] (the even CTA's are the ones used)
  uint64_t* empty = bars + kStages;       // [kStages]
  uint64_t* acc_full = empty + kStages;   // [2]
  uint64_t* acc_empty = acc_full + 2;     // [2] (the even CTA's are the ones used)
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? uniform(cluster_ctarank()) : 0u;
  constexpr int kUnit = C::kCluster;  // CTAs per tile
  const int unit = static_cast<int>(blockIdx.x) / kUnit;
  const int units = static_cast<int>(gridDim.x) / kUnit;
  const int total = p.tiles * p.batch;
  // this CTA's K blocks
  const int quarter_k = SPLIT ? uniform(cluster_ctarank()) : 0;
  const int kb0 = SPLIT ? p.k_blk * quarter_k / kSplitCtas : 0;
  const int kb1 = SPLIT ? p.k_blk * (quarter_k + 1) / kSplitCtas : p.k_blk;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], C::kEpiWarps * kCtas);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    if (PAIR) {
      tmem_alloc_pair(tmem_slot, kCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, kCols);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync();  // the peer's barriers exist before any remote signal
  tc_fence_after();
  const uint32_t tmem_base = uniform(*tmem_slot);

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    uint32_t stage = 0, phase = 1;  // parity of `empty` that a first use finds complete
    uint32_t loads = 0;
    bool ok = true;
    const uint32_t base = smem_addr(smem);
    // the even CTA's barrier, as a cluster address
    const uint32_t full0 = PAIR ? uniform(mapa_shared(smem_addr(full), 0)) : 0u;
    grid_dependency_wait();
    for (int t = unit; ok && t < total; t += units) {
      const int bi = t / p.tiles;
      int mi, ni;
      tile_of(p, t - bi * p.tiles, mi, ni);
      const int a_row = uniform((mi * kCtas + static_cast<int>(rank)) * 128);
      const int b_row = uniform(ni * kN + static_cast<int>(rank) * 128);
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!(ok = uniform_wait(&empty[stage], phase, abort_flag, p.status))) break;
        if (rank == 0) expect_tx_elected(&full[stage], kCtas * kStageBytes);
        const uint32_t a_dst = base + stage * kStageBytes, b_dst = a_dst + C::kABytes;
        const int k = 64 * kb;
        if (PAIR) {
          const uint32_t fb = full0 + stage * 8;
          tma_load_3d_pair_elected(&tmA, fb, a_dst, k, a_row, bi);
          if (B_MN) {
            tma_load_3d_pair_elected(&tmB, fb, b_dst, b_row, k, bi);
            tma_load_3d_pair_elected(&tmB, fb, b_dst + kBox, b_row + 64, k, bi);
          } else {
            tma_load_3d_pair_elected(&tmB, fb, b_dst, k, b_row, bi);
          }
        } else {
          tma_load_3d_elected(&tmA, &full[stage], a_dst, k, a_row, bi);
          if (B_MN) {
            tma_load_3d_elected(&tmB, &full[stage], b_dst, b_row, k, bi);
            tma_load_3d_elected(&tmB, &full[stage], b_dst + kBox, b_row + 64, k, bi);
          } else {
            tma_load_3d_elected(&tmB, &full[stage], b_dst, k, b_row, bi);
          }
        }
        ++loads;
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    // every stage this warp loaded has landed (the odd CTA's loads land on the
    // even CTA's barrier: it waits until the MMAs released them)
    if (lane == 0) {
      const uint32_t n_drain = loads < kStages ? loads : kStages;
      for (uint32_t i = 0; i < n_drain; ++i) {
        const uint32_t q = loads - 1 - i;
        mbar_wait_drain(rank == 0 ? &full[q % kStages] : &empty[q % kStages], (q / kStages) & 1);
      }
    }
  } else if (warp == 1) {
    // ----------------------------------------------------------------- MMA
    if (rank == 0) {
      uint32_t stage = 0, phase = 0, it = 0;
      bool ok = true;
      const Operand16 a_op(smem_addr(smem), 0), b_op(smem_addr(smem) + C::kABytes, B_MN ? kBox : 0);
      for (int t = unit; ok && t < total; t += units, ++it) {
        const uint32_t buf = it & 1, use = it >> 1;
        if (!uniform_wait(&acc_empty[buf], (use & 1) ^ 1, abort_flag, p.status)) break;
        tc_fence_after();
        const uint32_t d = tmem_base + buf * kN;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!(ok = uniform_wait(&full[stage], phase, abort_flag, p.status))) break;
          const Operand16 a = moved(a_op, stage * kStageBytes), b = moved(b_op, stage * kStageBytes);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t add = (kb > kb0 || k > 0) ? 1u : 0u;
            const uint32_t b_off = B_MN ? 2048 * k : 32 * k;
            if (PAIR)
              mma_f16_pair_at(d, a, 32 * k, b, b_off, kIdesc, add);
            else
              mma_f16_at(d, a, 32 * k, b, b_off, kIdesc, add);
          }
          if (PAIR)
            commit_pair_elected(&empty[stage], 0x3);
          else
            commit_elected(&empty[stage]);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        if (PAIR)
          commit_pair_elected(&acc_full[buf], 0x3);
        else
          commit_elected(&acc_full[buf]);
      }
      if (PAIR)
        commit_pair_elected(drain, 0x1);
      else
        commit_elected(drain);
      if (lane == 0) mbar_wait_drain(drain, 0);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    grid_dependency_wait();
    if (warp == 2 && lane == 0) grid_launch_dependents();
    const int q = warp & 3;
    const int part = (warp - 2) >> 2;  // of the tile's columns
    uint8_t* buf_s = staging + (warp - 2) * kStagingBytes;
    uint32_t it = 0;
    bool ok = false;  // SPLIT: the partial sum is complete
    for (int t = unit; t < total; t += units, ++it) {
      const uint32_t buf = it & 1, use = it >> 1;
      const int bi = t / p.tiles;
      int mi, ni;
      tile_of(p, t - bi * p.tiles, mi, ni);
      const int row0 = (mi * kCtas + static_cast<int>(rank)) * 128 + 32 * q;
      const int col0 = ni * kN + part * (kN / kParts);
      Addend<MODE> add;
      if (!SPLIT) add.fetch(p, bi, row0, col0);
      if (!uniform_wait(&acc_full[buf], use & 1, abort_flag, p.status)) break;
      tc_fence_after();
      if (SPLIT) {  // one tile per cluster: the rest comes after the loop
        ok = true;
        break;
      }
      epilogue<MODE>(p, add,
                     tmem_base + (static_cast<uint32_t>(32 * q) << 16) + buf * kN + part * (kN / kParts),
                     bi, row0, col0, kN / kParts, p.symmetric && mi != ni, buf_s);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (PAIR)
          mbar_arrive_cluster(mapa_shared(smem_addr(&acc_empty[buf]), 0));
        else
          mbar_arrive(&acc_empty[buf]);
      }
    }
    if (SPLIT) {
      // Every CTA's loads and MMAs are done (the other warps come here when they
      // are): its ring takes the partial sums for the 32 columns it finishes.
      const int row = 32 * q + lane;
      __syncwarp();
      cluster_sync();
      if (ok)
        send_partial(tmem_base + (static_cast<uint32_t>(32 * q) << 16) + part * 64, smem,
                     static_cast<uint32_t>(quarter_k), row, part);
      const int bi = unit / p.tiles;
      int mi, ni;
      tile_of(p, unit - bi * p.tiles, mi, ni);
      const int row0 = mi * 128 + 32 * q, col0 = ni * 128 + 32 * quarter_k;
      const bool mine = ok && part == 0 && row0 < p.rows && col0 < p.cols;
      Addend<MODE> add;
      if (mine) add.fetch(p, bi, row0, col0);
      __syncwarp();
      cluster_sync();
      if (mine) {
        float acc[32];
        sum_partials(smem, row, acc);
        finish_block<MODE>(p, add, acc, bi, row0, col0, p.symmetric && mi != ni, buf_s);
      }
    }
  }
  if (SPLIT && warp < 2) {  // the two barriers of the epilogue
    __syncwarp();
    cluster_sync();
    cluster_sync();
  }
  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync();  // neither CTA leaves while the pair still uses it
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    if (PAIR)
      tmem_dealloc_pair(tmem_base, kCols);
    else
      tmem_dealloc(tmem_base, kCols);
  }
}

// ------------------------------------------------- A^2 and the update at once
// For k <= 256, where A fits into shared memory: a CTA computes the 128 rows of
// B = b A + c A^2 that its 128 x 128 tile of X takes (again in every CTA of those
// rows: 1 us of products), puts them in the place of A's rows, and goes on with B X.
// That saves a launch, and X is fetched while the launch before still runs: eight
// 256 x 1024 104 -> 85 us, one 256 x 256 83 -> 65, 64 x 64 61 -> 51.
constexpr int kSmallK = 256;
constexpr int kSmallWarps = 16;  // as in Config<kSingle>
constexpr int kSmallThreads = 64 + 32 * kSmallWarps;
constexpr uint32_t kABox = 128 * 128;   // 128 rows x 64 fp16
constexpr uint32_t kXBlock = 2 * kBox;  // 64 rows x 128 fp16, as two boxes
constexpr uint32_t kSmallSmem = 1024 + 8 * kABox + 4 * kXBlock + 256;
static_assert(kSmallWarps * kStagingBytes <= 4 * kXBlock, "the last stage uses X's place");

__global__ void __launch_bounds__(kSmallThreads, 1)
    ortho_small_update(const __grid_constant__ CUtensorMap tmA,
                       const __grid_constant__ CUtensorMap tmX, const OrthoParams p) {
  constexpr uint32_t kIdescSquare = make_idesc(0, false, false, 128, 128);
  constexpr uint32_t kIdescUpdate = make_idesc(0, false, true, 128, 128);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* smA = smem;               // [K block][row half] boxes
  uint8_t* smX = smem + 8 * kABox;   // [K block]
  uint64_t* a_full = reinterpret_cast<uint64_t*>(smX + 4 * kXBlock);
  uint64_t* x_full = a_full + 1;
  uint64_t* square_full = a_full + 2;
  uint64_t* b_full = a_full + 3;
  uint64_t* acc_full = a_full + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(a_full + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int bi = static_cast<int>(blockIdx.x) / p.tiles, t = static_cast<int>(blockIdx.x) % p.tiles;
  const int mi = t % p.m_blk, ni = t / p.m_blk;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 5; ++i) mbar_init(&a_full[i], i == 3 ? kSmallWarps : 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t square = uniform(*tmem_slot), acc = square + kSmallK;  // 256 and 128 columns

  // The launch before (A = X X^T) let this one start when it had waited for the
  // launch that made X: X is complete.  A is, once this launch has waited.
  if (warp == 0) {
    expect_tx_elected(x_full, p.k_blk * kXBlock);
    for (int kb = 0; kb < p.k_blk; ++kb)
      for (int c = 0; c < 2; ++c)
        tma_load_3d_elected(&tmX, x_full, smem_addr(smX) + kb * kXBlock + c * kBox,
                            128 * ni + 64 * c, 64 * kb, bi);
    grid_dependency_wait();
    expect_tx_elected(a_full, p.k_blk * p.m_blk * kABox);
    for (int kb = 0; kb < p.k_blk; ++kb)
      for (int r = 0; r < p.m_blk; ++r)
        tma_load_3d_elected(&tmA, a_full, smem_addr(smA) + (2 * kb + r) * kABox, 64 * kb, 128 * r,
                            bi);
    if (lane == 0) {  // every load has landed before this CTA's shared memory goes away
      mbar_wait_drain(x_full, 0);
      mbar_wait_drain(a_full, 0);
    }
  } else if (warp == 1) {
    const Operand16 a_op(smem_addr(smA), 0), x_op(smem_addr(smX), kBox);
    if (uniform_wait(a_full, 0, abort_flag, p.status)) {
      tc_fence_after();
      for (int r = 0; r < p.m_blk; ++r)
        for (int kb = 0; kb < p.k_blk; ++kb) {
          const Operand16 a = moved(a_op, (2 * kb + mi) * kABox), b = moved(a_op, (2 * kb + r) * kABox);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_f16_at(square + 128 * r, a, 32 * k, b, 32 * k, kIdescSquare,
                       (kb > 0 || k > 0) ? 1u : 0u);
        }
      commit_elected(square_full);
    }
    if (uniform_wait(x_full, 0, abort_flag, p.status) &&
        uniform_wait(b_full, 0, abort_flag, p.status)) {
      tc_fence_after();
      for (int kb = 0; kb < p.k_blk; ++kb) {
        const Operand16 b = moved(a_op, (2 * kb + mi) * kABox), x = moved(x_op, kb * kXBlock);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_f16_at(acc, b, 32 * k, x, 2048 * k, kIdescUpdate, (kb > 0 || k > 0) ? 1u : 0u);
      }
    }
    commit_elected(acc_full);  // all MMAs issued by this thread are done
    if (lane == 0) mbar_wait_drain(acc_full, 0);
  } else {
    const int q = warp & 3, part = (warp - 2) >> 2;
    const uint32_t lanes = static_cast<uint32_t>(32 * q) << 16;
    const int row0 = mi * 128 + 32 * q, col0 = ni * 128 + 32 * part;
    Addend<kUpdate> add;
    add.fetch(p, bi, row0, col0);
    grid_dependency_wait();  // nothing is stored before the launch before is complete
    if (warp == 2 && lane == 0) grid_launch_dependents();
    bool ok = uniform_wait(square_full, 0, abort_flag, p.status);
    if (ok && part < p.k_blk) {
      // K block `part` of B's rows, in the place of A's
      tc_fence_after();
      const int row = 32 * q + lane;
      const uint8_t* mine = smA + (2 * part + mi) * kABox + row * 128;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t r[32];
        tmem_ld_32x32b_x32(square + lanes + 64 * part + 32 * u, r);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t at = ((4 * u + i) ^ (row & 7)) << 4;
          const uint4 a = *reinterpret_cast<const uint4*>(mine + at);
          const uint32_t w[4] = {a.x, a.y, a.z, a.w};
          uint32_t o[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
            o[k] = pack_half2(
                fmaf(p.c * kUnhold, __uint_as_float(r[8 * i + 2 * k]), p.b * f.x),
                fmaf(p.c * kUnhold, __uint_as_float(r[8 * i + 2 * k + 1]), p.b * f.y));
          }
          st_shared_v4(smem_addr(mine) + at, o[0], o[1], o[2], o[3]);
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(b_full);
    ok = uniform_wait(acc_full, 0, abort_flag, p.status) && ok;
    if (ok && row0 < p.rows && col0 < p.cols) {
      tc_fence_after();
      uint32_t r[32];
      tmem_ld_32x32b_x32(acc + lanes + 32 * part, r);
      tmem_ld_wait();
      // X's place stages the stores: every MMA is done
      finish_block<kUpdate>(p, add, reinterpret_cast<const float(&)[32]>(r), bi, row0, col0, false,
                            smX + (warp - 2) * kStagingBytes);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(square, 512);
  }
}

// ------------------------------------------------------------- norm and split
constexpr int kNormThreads = 256;
constexpr int kMaxParts = 256;  // partial sums of one matrix (kNormThreads at most)

template <int ELT>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  return ELT == 4 ? static_cast<const float*>(p)[i]
                  : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i])
                                    << 16);
}

// Sum over the CTA in a fixed order, in every thread.
__device__ float cta_sum(float s) {
  __shared__ float part[kNormThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
  __syncthreads();
  float all = 0.f;
#pragma unroll
  for (int w = 0; w < kNormThreads / 32; ++w) all += part[w];
  __syncthreads();
  return all;
}

// The largest |x| over the CTA, in every thread.
__device__ float cta_max(float x) {
  __shared__ float part[kNormThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
  __syncthreads();
  float all = 0.f;
#pragma unroll
  for (int w = 0; w < kNormThreads / 32; ++w) all = fmaxf(all, part[w]);
  __syncthreads();
  return all;
}

// A sum of squares: 4^exponent times sum.
struct Part {
  float sum;
  int32_t exponent;
};

// Squares below 2^-126 lose bits, and those of 2^40 elements lose less than 2^-109 in
// all; a sum of this and more, and finite, is as good as fp32 makes it.
constexpr float kSumLow = 0x1p-80f;

// f(element) for the elements of this thread's share of a matrix, in order.
template <int ELT, class F>
__device__ __forceinline__ void for_share(const void* g, int64_t elems, int vec, F f) {
  const int64_t base = static_cast<int64_t>(blockIdx.y) * elems;
  const int64_t me = static_cast<int64_t>(blockIdx.x) * kNormThreads + threadIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kNormThreads;
  if (vec) {
    constexpr int kPer = 16 / ELT;
    const uint4* v = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(g) + base * ELT);
    const int64_t n = elems / kPer;
#pragma unroll 4
    for (int64_t i = me; i < n; i += step) {
      const uint4 q = __ldg(v + i);
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (ELT == 4) {
          f(__uint_as_float(w[k]));
        } else {
          f(__uint_as_float(w[k] << 16));
          f(__uint_as_float(w[k] & 0xffff0000u));
        }
      }
    }
  } else {
#pragma unroll 4
    for (int64_t i = me; i < elems; i += step) f(load1<ELT>(g, base + i));
  }
}

// The sum of squares of a share whose plain sum was not: each element scaled by a power
// of two that takes the largest to about 1, and added in the same order, so that a power
// of two in G changes nothing else.
template <int ELT>
__device__ __noinline__ Part scaled_sum(const void* g, int64_t elems, int vec) {
  float top = 0.f;
  for_share<ELT>(g, elems, vec, [&](float x) { top = fmaxf(top, fabsf(x)); });
  top = cta_max(top);
  if (!(top > 0.f) || isinf(top)) return Part{top, 0};
  int e = ilogbf(top);
  e = e < -126 ? -126 : e > 126 ? 126 : e;  // 2^-e is exact
  const float f = ldexpf(1.f, -e);
  float s = 0.f;
  for_share<ELT>(g, elems, vec, [&](float x) { s = fmaf(x * f, x * f, s); });
  return Part{cta_sum(s), e};
}

// parts[b][x] = sum of squares of the x-th share of matrix b.
template <int ELT>
__global__ void __launch_bounds__(kNormThreads)
    ortho_norm(const void* g, int64_t elems, int vec, Part* parts) {
  grid_launch_dependents();
  float s = 0.f;
  for_share<ELT>(g, elems, vec, [&](float x) { s = fmaf(x, x, s); });
  Part part{cta_sum(s), 0};
  if (part.sum < kSumLow || isinf(part.sum))  // the same in every thread
    part = scaled_sum<ELT>(g, elems, vec);
  if (threadIdx.x == 0) parts[static_cast<int64_t>(blockIdx.y) * kMaxParts + blockIdx.x] = part;
}

struct SplitParams {
  const void* g;
  int64_t rows, cols;      // of G
  const Part* parts;
  int32_t n_parts;
  float eps;
  float* x;                // [k][ldx]
  __half* xh;              // [k][ldh]
  int64_t ldx, ldh, x_stride, h_stride;
};

// X = G * scale * inverse, from the partial sums of the launch before.
struct Normal {
  float scale;    // a power of two: 1 unless |G_b| is far from it
  float inverse;  // 1 / ((|G_b| + eps) * scale)
  __device__ __forceinline__ float operator()(float g) const { return g * scale * inverse; }
};

__device__ Normal normal_of(const SplitParams& p, int b) {
  grid_dependency_wait();
  grid_launch_dependents();
  constexpr int kNone = -1000;
  Part part{0.f, kNone};
  if (threadIdx.x < p.n_parts) {
    part = p.parts[static_cast<int64_t>(b) * kMaxParts + threadIdx.x];
    if (part.sum == 0.f) part.exponent = kNone;  // zeros are of any scale
  }
  __shared__ int exponent;
  if (threadIdx.x == 0) exponent = kNone;
  __syncthreads();
  const int e = __reduce_max_sync(0xffffffffu, part.exponent);
  if ((threadIdx.x & 31) == 0) atomicMax(&exponent, e);
  __syncthreads();
  const int top = exponent == kNone ? 0 : exponent;
  if (part.exponent != kNone && part.exponent != top)
    part.sum = ldexpf(part.sum, 2 * (part.exponent - top));
  const float scale = ldexpf(1.f, -top);
  return Normal{scale, 1.f / (sqrtf(cta_sum(part.sum)) + p.eps * scale)};
}

// X = G / (|G| + eps) in fp32 and, times 4096, in fp16, for G with rows of
// whole 16-byte vectors and rows <= cols: eight elements per thread at a time.
template <int ELT>
__global__ void __launch_bounds__(kNormThreads) ortho_split_rows(const SplitParams p) {
  const int b = static_cast<int>(blockIdx.y);
  const Normal normal = normal_of(p, b);
  const uint8_t* g = static_cast<const uint8_t*>(p.g) + static_cast<int64_t>(b) * p.rows * p.cols * ELT;
  const int64_t per_row = p.ldx / 8, n = p.rows * per_row;
#pragma unroll 2
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kNormThreads + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * kNormThreads) {
    const int64_t r = i / per_row, c = (i - r * per_row) * 8;
    float v[8] = {};
    if (c < p.cols) {
      const uint4* src = reinterpret_cast<const uint4*>(g + (r * p.cols + c) * ELT);
      if (ELT == 4) {
        const uint4 lo = __ldcs(src), hi = __ldcs(src + 1);
        const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(w[k]);
      } else {
        const uint4 q = __ldcs(src);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          v[2 * k] = __uint_as_float(w[k] << 16);
          v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = normal(v[k]);
    float4* x = reinterpret_cast<float4*>(p.x + b * p.x_stride + r * p.ldx + c);
    x[0] = make_float4(v[0], v[1], v[2], v[3]);
    x[1] = make_float4(v[4], v[5], v[6], v[7]);
    uint32_t h[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) h[k] = pack_half2(v[2 * k] * kHold, v[2 * k + 1] * kHold);
    *reinterpret_cast<uint4*>(p.xh + b * p.h_stride + r * p.ldh + c) =
        make_uint4(h[0], h[1], h[2], h[3]);
  }
}

// The same for any G, in 64 x 64 blocks, which TRANSPOSED turns around in
// shared memory.
template <int ELT, bool TRANSPOSED>
__global__ void __launch_bounds__(kNormThreads) ortho_split(const SplitParams p) {
  __shared__ float tile[TRANSPOSED ? 64 : 1][65];
  const int b = static_cast<int>(blockIdx.z);
  const Normal normal = normal_of(p, b);
  const int64_t base = static_cast<int64_t>(b) * p.rows * p.cols;
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * 64, c0 = static_cast<int64_t>(blockIdx.x) * 64;
  float* x = p.x + b * p.x_stride;
  __half* xh = p.xh + b * p.h_stride;
  const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;  // 64 x 4
  if (TRANSPOSED) {
#pragma unroll
    for (int i = 0; i < 64; i += 4) {
      const int64_t r = r0 + ty + i, c = c0 + tx;
      tile[ty + i][tx] = (r < p.rows && c < p.cols) ? load1<ELT>(p.g, base + r * p.cols + c) : 0.f;
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 64; i += 4) {
    // row and column of X (k x n)
    const int64_t r = (TRANSPOSED ? c0 : r0) + ty + i, c = (TRANSPOSED ? r0 : c0) + tx;
    const int64_t k = TRANSPOSED ? p.cols : p.rows, n = TRANSPOSED ? p.rows : p.cols;
    if (r >= k) continue;
    float v = 0.f;
    if (c < n) v = normal(TRANSPOSED ? tile[tx][ty + i] : load1<ELT>(p.g, base + r * p.cols + c));
    if (c < p.ldx) x[r * p.ldx + c] = v;
    if (c < p.ldh) xh[r * p.ldh + c] = __float2half_rn(v * kHold);
  }
}

// --------------------------------------------------------------------- host
// The singular values of X start in [0, 1] and each step takes s to
// p(s) = s (a + b s^2 + c s^4).  Bounds |s| over the steps by p's values at the
// ends of the interval and at its turning points; false if |s|, or an
// eigenvalue b s^2 + c s^4 of B, or s^2 leaves the range fp16 holds here.
bool check_polynomial(double a, double b, double c, int steps) {
  if (!(std::isfinite(a) && std::isfinite(b) && std::isfinite(c))) return false;
  double top = 1.0;
  for (int i = 0; i < steps; ++i) {
    const double t = top * top;  // s^2 in [0, t]
    double eig = std::fabs(b * t + c * t * t);
    if (c != 0.0) {
      const double v = -b / (2 * c);
      if (v > 0 && v < t) eig = std::fmax(eig, std::fabs(b * v + c * v * v));
    }
    if (!(eig < 15.0) || !(t < 15.0)) return false;
    auto value = [&](double s2) { return std::fabs(std::sqrt(s2) * (a + b * s2 + c * s2 * s2)); };
    double next = value(t);
    // p'(s) = a + 3 b s^2 + 5 c s^4 = 0
    if (c != 0.0) {
      const double disc = 9 * b * b - 20 * a * c;
      if (disc >= 0) {
        for (int sign = -1; sign <= 1; sign += 2) {
          const double r = (-3 * b + sign * std::sqrt(disc)) / (10 * c);
          if (r > 0 && r < t) next = std::fmax(next, value(r));
        }
      }
    } else if (b != 0.0) {
      const double r = -a / (3 * b);
      if (r > 0 && r < t) next = std::fmax(next, value(r));
    }
    top = next * 1.001;  // rounding of the operands
    if (!(top < 3.8)) return false;
  }
  return true;
}

struct Layout {
  int64_t k, n, ldx, ldh, lda;
  int32_t parts;
  size_t off_parts, off_x, off_h[2], off_a, off_b, total;
};

Layout layout(int64_t batch, int64_t rows, int64_t cols) {
  Layout l{};
  l.k = rows < cols ? rows : cols;
  l.n = rows < cols ? cols : rows;
  l.ldx = (l.n + 63) / 64 * 64;
  l.ldh = l.ldx;
  l.lda = (l.k + 63) / 64 * 64;
  const int64_t elems = rows * cols;
  int64_t parts = (elems + 8191) / 8192;
  l.parts = static_cast<int32_t>(parts < 1 ? 1 : parts > kMaxParts ? kMaxParts : parts);
  size_t o = 0;
  const size_t B = static_cast<size_t>(batch);
  l.off_parts = o;
  o += round256(B * kMaxParts * sizeof(Part));
  l.off_x = o;
  o += round256(B * static_cast<size_t>(l.k * l.ldx) * 4);
  for (int i = 0; i < 2; ++i) {
    l.off_h[i] = o;
    o += round256(B * static_cast<size_t>(l.k * l.ldh) * 2);
  }
  l.off_a = o;
  o += round256(B * static_cast<size_t>(l.k * l.lda) * 2);
  l.off_b = o;
  o += round256(B * static_cast<size_t>(l.k * l.lda) * 2);
  l.total = o;
  return l;
}

// An fp16 [batch][rows][cols] operand; box of 64 columns by `box_rows`.
int half_map(CUtensorMap* m, const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t stride,
             int64_t batch, uint32_t box_rows, const char* what) {
  const uint64_t dims[3] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(rows),
                            static_cast<uint64_t>(batch)};
  const uint64_t pitch[2] = {static_cast<uint64_t>(ld) * 2, static_cast<uint64_t>(stride) * 2};
  const uint32_t box[3] = {64, box_rows, 1};
  return host_tensor_map(m, p, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, dims, pitch, box, what);
}

template <int MODE, Shape SHAPE>
cudaError_t launch_shape(const CUtensorMap& A, const CUtensorMap& B, OrthoParams p, int64_t k,
                         int sms, cudaStream_t s) {
  using C = Config<SHAPE>;
  p.m_blk = (p.rows + C::kM - 1) / C::kM;
  p.n_blk = (p.cols + C::kN - 1) / C::kN;
  p.k_blk = static_cast<int32_t>((k + 63) / 64);
  p.symmetric = MODE != kUpdate;
  p.tiles = p.symmetric ? p.m_blk * (p.m_blk + 1) / 2 : p.m_blk * p.n_blk;
  const auto kernel = ortho_gemm<MODE, SHAPE>;
  static SmemLimit limit;
  const cudaError_t e = limit.raise(kernel, C::kSmem);
  if (e != cudaSuccess) return e;
  const int64_t total = static_cast<int64_t>(p.tiles) * p.batch;
  const int64_t cap = SHAPE == kSplit ? total : sms / C::kCluster;  // split: one tile each
  const int64_t units = total < cap ? total : cap;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cfg.gridDim = dim3(static_cast<unsigned>(units * C::kCluster));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C::kCluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  // the prologue overlaps the previous launch's tail; loads and stores wait
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, A, B, p);
}

// Rounds of tiles, whose epilogues run beside the next round's products, and one
// epilogue at the end.  Times in units of 0.03 us: a K block of 64 takes 7 on a 128 x
// 128 tile (L2 feeds all SMs at 21 TB/s) and 10 on a pair's 256 x 256; an epilogue 2.5
// us and 4.5, a pair's update 6.5.
int64_t round_time(int64_t tiles, int64_t at_once, int64_t products, int64_t epilogue) {
  return (tiles + at_once - 1) / at_once * (products > epilogue ? products : epilogue) + epilogue;
}

// X X^T by four CTAs per 128 x 128 tile, where the GPU has that many and K is at least
// 2048 (300 x 8000 all told 159 us against 226, 1000 x 3584 187 against 199, 512 x 2048
// 123 against 128; but 1024 x 1024 157 against 130: the exchange of the partial sums
// takes about 5 us).  The other products have such a K only where they have more tiles.
// Else the shape that the estimate above favours.  All told, single CTAs against pairs:
// 3000 x 3000 479 us against 576 (78 pairs of tiles on 76 pairs of SMs), 1024 x 16000
// 414 against 435, 1500 x 4000 260 against 281, 16 of 384 x 2000 261 against 309; but
// 2304 x 2304 363 against 348, 4096 x 4096 1154 against 1034.
Shape gemm_shape(int mode, int64_t rows, int64_t cols, int64_t k, int64_t batch, int sms) {
  auto tiles = [&](int64_t edge) {
    const int64_t mb = (rows + edge - 1) / edge, nb = (cols + edge - 1) / edge;
    return (mode != kUpdate ? mb * (mb + 1) / 2 : mb * nb) * batch;
  };
  if (mode == kGram && tiles(128) * kSplitCtas <= sms && k >= 2048) return kSplit;
  const int64_t k_blk = (k + 63) / 64;
  return round_time(tiles(128), sms, 7 * k_blk, 83) <=
                 round_time(tiles(256), sms / 2, 10 * k_blk, mode == kUpdate ? 217 : 150)
             ? kSingle
             : kPair;
}

template <int MODE>
cudaError_t launch_gemm(const CUtensorMap& A, const CUtensorMap& B, const OrthoParams& p, int64_t k,
                        int sms, cudaStream_t s) {
  const Shape shape = gemm_shape(MODE, p.rows, p.cols, k, p.batch, sms);
  if constexpr (MODE == kGram) {
    if (shape == kSplit) return launch_shape<MODE, kSplit>(A, B, p, k, sms, s);
  }
  return shape == kSingle ? launch_shape<MODE, kSingle>(A, B, p, k, sms, s)
                          : launch_shape<MODE, kPair>(A, B, p, k, sms, s);
}

// A launch that may start while the one before finishes; the kernel waits for it.
template <class... ARGS>
cudaError_t launch_after(void (*kernel)(ARGS...), dim3 grid, int threads, uint32_t smem,
                         cudaStream_t s, const ARGS&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Up to two rounds of CTAs (300 of 64 x 64 170 -> 92 us, 256 x 16000 182 -> 179; but
// 256 x 65536 545 -> 611: there the tiles' loads, products and stores should overlap).
bool small_update(int64_t rows, int64_t cols, int64_t batch, int sms) {
  return rows <= kSmallK && (rows + 127) / 128 * ((cols + 127) / 128) * batch <= 2 * sms;
}

cudaError_t launch_small_update(const CUtensorMap& A, const CUtensorMap& X, OrthoParams p,
                                cudaStream_t s) {
  static SmemLimit limit;
  const cudaError_t e = limit.raise(ortho_small_update, kSmallSmem);
  if (e != cudaSuccess) return e;
  p.m_blk = (p.rows + 127) / 128;
  p.n_blk = (p.cols + 127) / 128;
  p.k_blk = (p.rows + 63) / 64;
  p.tiles = p.m_blk * p.n_blk;
  return launch_after(ortho_small_update, dim3(static_cast<unsigned>(p.tiles * p.batch)),
                      kSmallThreads, kSmallSmem, s, A, X, p);
}

int run(const void* g, int32_t dtype, int64_t batch, int64_t rows, int64_t cols, int steps,
        const float* coeffs, float eps, void* out, const Layout& l, uint8_t* w, int32_t* status,
        int sms, cudaStream_t s) {
  Part* parts = reinterpret_cast<Part*>(w + l.off_parts);
  float* x = reinterpret_cast<float*>(w + l.off_x);
  __half* h[2] = {reinterpret_cast<__half*>(w + l.off_h[0]),
                  reinterpret_cast<__half*>(w + l.off_h[1])};
  __half* A = reinterpret_cast<__half*>(w + l.off_a);
  __half* Bm = reinterpret_cast<__half*>(w + l.off_b);
  const int64_t elems = rows * cols;
  const int elt = dtype == FLCE_FP32 ? 4 : 2;
  const int vec = aligned16(g) && (elems * elt) % 16 == 0;
  const unsigned nb = static_cast<unsigned>(batch);
  const dim3 ngrid(static_cast<unsigned>(l.parts), nb);
  if (elt == 4)
    ortho_norm<4><<<ngrid, kNormThreads, 0, s>>>(g, elems, vec, parts);
  else
    ortho_norm<2><<<ngrid, kNormThreads, 0, s>>>(g, elems, vec, parts);
  FLCE_TRY(cudaGetLastError());
  const SplitParams sp{g,   rows, cols,  parts, l.parts,      eps,
                       x,   h[0], l.ldx, l.ldh, l.k * l.ldx,  l.k * l.ldh};
  const bool tr = rows > cols;
  if (!tr && aligned16(g) && cols % 8 == 0) {
    const int64_t want = (l.k * (l.ldx / 8) + kNormThreads - 1) / kNormThreads, cap = 8 * sms;
    const dim3 sgrid(static_cast<unsigned>(want < cap ? want : cap), nb);
    FLCE_TRY(launch_after(elt == 4 ? ortho_split_rows<4> : ortho_split_rows<2>, sgrid,
                          kNormThreads, 0, s, sp));
  } else {
    const dim3 sgrid(static_cast<unsigned>((cols + 63) / 64),
                     static_cast<unsigned>((rows + 63) / 64), nb);
    FLCE_TRY(launch_after(elt == 4 ? (tr ? ortho_split<4, true> : ortho_split<4, false>)
                                   : (tr ? ortho_split<2, true> : ortho_split<2, false>),
                          sgrid, kNormThreads, 0, s, sp));
  }
  int rc;
  CUtensorMap mx[2], mxn[2], ma, mb;
  for (int i = 0; i < 2; ++i) {
    if ((rc = half_map(&mx[i], h[i], l.k, l.n, l.ldh, l.k * l.ldh, batch, 128, "X"))) return rc;
    if ((rc = half_map(&mxn[i], h[i], l.k, l.n, l.ldh, l.k * l.ldh, batch, 64, "X^T"))) return rc;
  }
  if ((rc = half_map(&ma, A, l.k, l.k, l.lda, l.k * l.lda, batch, 128, "A"))) return rc;
  if ((rc = half_map(&mb, Bm, l.k, l.k, l.lda, l.k * l.lda, batch, 128, "B"))) return rc;
  OrthoParams p{};
  p.batch = static_cast<int32_t>(batch);
  p.rows = static_cast<int32_t>(l.k);
  p.x = x;
  p.ldx = l.ldx;
  p.x_stride = l.k * l.ldx;
  p.a = coeffs[0];
  p.b = coeffs[1];
  p.c = coeffs[2];
  p.status = status;
  for (int i = 0; i < steps; ++i) {
    p.cols = static_cast<int32_t>(l.k);
    p.ld = l.lda;
    p.stride = l.k * l.lda;
    p.out = A;
    FLCE_TRY(launch_gemm<kGram>(mx[i & 1], mx[i & 1], p, l.n, sms, s));
    OrthoParams poly = p;
    poly.out = Bm;
    poly.gram = A;
    p.cols = static_cast<int32_t>(l.n);
    p.ld = l.ldh;
    p.stride = l.k * l.ldh;
    p.out = h[(i + 1) & 1];
    if (i == steps - 1) {
      p.result = static_cast<uint16_t*>(out);
      p.transposed = tr;
      p.result_vec = aligned16(out) && cols % 8 == 0;
    }
    if (small_update(p.rows, p.cols, p.batch, sms)) {
      FLCE_TRY(launch_small_update(ma, mxn[i & 1], p, s));
      continue;
    }
    FLCE_TRY(launch_gemm<kPoly>(ma, ma, poly, l.k, sms, s));
    FLCE_TRY(launch_gemm<kUpdate>(mb, mxn[i & 1], p, l.k, sms, s));
  }
  return FLCE_OK;
}

}  // namespace
}  // namespace flce

using namespace flce;

extern "C" int flce_orthogonalize(const void* G, int64_t batch, int64_t rows, int64_t cols,
                                  int32_t steps, const float* coeffs, float eps, void* out,
                                  const flce_opts* opts) {
  host_clear_error();
  const flce_opts o = opts_or_default(opts);
  if (o.dtype != FLCE_BF16 && o.dtype != FLCE_FP32)
    return host_error(FLCE_ERR_ARG, "flce_orthogonalize: unknown dtype %d", o.dtype);
  if (batch < 0 || rows < 0 || cols < 0 || batch > 65535 || rows > (1 << 20) || cols > (1 << 20))
    return host_error(FLCE_ERR_ARG,
                      "flce_orthogonalize: 0 <= batch <= 65535 and 0 <= rows, cols <= 2^20");
  if (steps < 1 || steps > 64)
    return host_error(FLCE_ERR_ARG, "flce_orthogonalize: steps must be in 1 .. 64");
  if (!(eps >= 0.f) || std::isinf(eps))
    return host_error(FLCE_ERR_ARG, "flce_orthogonalize: eps must be finite and not negative");
  const float standard[3] = {3.4445f, -4.7750f, 2.0315f};
  const float* c = coeffs ? coeffs : standard;
  if (!check_polynomial(c[0], c[1], c[2], steps))
    return host_error(FLCE_ERR_ARG,
                      "flce_orthogonalize: the polynomial takes singular values of [0, 1] out of "
                      "the range of the fp16 products");
  const bool empty = batch == 0 || rows == 0 || cols == 0;
  if (!empty && (!G || !out)) return host_error(FLCE_ERR_ARG, "flce_orthogonalize: null pointer");
  const uintptr_t el = o.dtype == FLCE_FP32 ? 3 : 1;
  if ((reinterpret_cast<uintptr_t>(G) & el) || (reinterpret_cast<uintptr_t>(out) & 1))
    return host_error(FLCE_ERR_ALIGN, "flce_orthogonalize: misaligned pointer");
  int sms = 0;
  int rc = host_device(&sms);
  if (rc) return rc;
  const Layout l = layout(batch, rows, cols);
  const int64_t blocks = (l.k + 127) / 128 * ((l.n + 127) / 128) * batch;
  if (blocks >= (int64_t{1} << 31) || (rows + 63) / 64 > 65535)
    return host_error(FLCE_ERR_ARG, "flce_orthogonalize: too many tiles");
  StepCall call;
  if ((rc = call.begin(o, empty ? 0 : l.total, empty ? StepCall::kIfAsked : StepCall::kCleared)))
    return rc;
  if (!empty)
    rc = run(G, o.dtype, batch, rows, cols, steps, c, eps, out, l, call.scratch, call.status, sms,
             call.stream);
  return call.end(rc);
}

extern "C" int flce_selftest_ortho_shapes(int64_t batch, int64_t rows, int64_t cols, int32_t sms,
                                          int32_t shapes[3]) {
  host_clear_error();
  if (batch < 1 || rows < 1 || cols < 1 || batch > 65535 || rows > (1 << 20) ||
      cols > (1 << 20) || sms < 2 || !shapes)
    return host_error(FLCE_ERR_ARG, "flce_selftest_ortho_shapes: sizes out of range");
  const Layout l = layout(batch, rows, cols);
  const bool merged = small_update(l.k, l.n, batch, sms);
  shapes[0] = gemm_shape(kGram, l.k, l.k, l.n, batch, sms);
  shapes[1] = merged ? 3 : gemm_shape(kPoly, l.k, l.k, l.k, batch, sms);
  shapes[2] = merged ? 3 : gemm_shape(kUpdate, l.k, l.n, l.k, batch, sms);
  return FLCE_OK;
}
