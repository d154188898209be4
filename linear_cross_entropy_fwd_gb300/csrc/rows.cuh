// rows.cuh -- rows of activations in registers: octets (8 consecutive elements) of bf16 or
// fp32, and sums over the warps that share a row.
#pragma once
#include "sm103.cuh"

namespace flce {

struct bf16_t {};  // element tags; fp32 is `float`

template <class T>
struct Elem;
template <>
struct Elem<bf16_t> {
  static constexpr int kBytes = 2;
  using Octet = uint4;
};
template <>
struct Elem<float> {
  static constexpr int kBytes = 4;
  struct Octet {
    uint4 a, b;
  };
};

__device__ __forceinline__ void octet_floats(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void octet_floats(const Elem<float>::Octet& v, float (&f)[8]) {
  const uint32_t w[8] = {v.a.x, v.a.y, v.a.z, v.a.w, v.b.x, v.b.y, v.b.z, v.b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
}

__device__ __forceinline__ uint4 to_octet(bf16_t, const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ Elem<float>::Octet to_octet(float, const float (&f)[8]) {
  Elem<float>::Octet o;
  o.a = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                   __float_as_uint(f[3]));
  o.b = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]),
                   __float_as_uint(f[7]));
  return o;
}

// Octet `o` of a row of T at `row`.
template <class T>
__device__ __forceinline__ typename Elem<T>::Octet load_octet(const void* row, int o) {
  return static_cast<const typename Elem<T>::Octet*>(row)[o];
}
template <class T>
__device__ __forceinline__ void store_octet(void* row, int o, const float (&f)[8]) {
  static_cast<typename Elem<T>::Octet*>(row)[o] = to_octet(T{}, f);
}

template <class T>
__device__ __forceinline__ const void* row_at(const void* base, int64_t row, int64_t stride) {
  return static_cast<const uint8_t*>(base) + row * stride * Elem<T>::kBytes;
}
template <class T>
__device__ __forceinline__ void* row_at(void* base, int64_t row, int64_t stride) {
  return static_cast<uint8_t*>(base) + row * stride * Elem<T>::kBytes;
}

// Octet `o` of a parameter vector, fp32 or T; `missing` for each element without a vector.
template <class T>
__device__ __forceinline__ void param_octet(const void* p, bool fp32, int o, float missing,
                                            float (&f)[8]) {
  if (!p) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = missing;
  } else if (fp32) {
    octet_floats(load_octet<float>(p, o), f);
  } else {
    octet_floats(load_octet<T>(p, o), f);
  }
}

// One element of type T, or fp32.
template <class T>
__device__ __forceinline__ float one_element(const void* p, bool fp32, int64_t i) {
  if (fp32 || Elem<T>::kBytes == 4) return static_cast<const float*>(p)[i];
  return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << 16);
}
__device__ __forceinline__ void store_element(bf16_t, void* p, int64_t i, float v) {
  static_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(pack_bf16x2(v, 0.f));
}
__device__ __forceinline__ void store_element(float, void* p, int64_t i, float v) {
  static_cast<float*>(p)[i] = v;
}

__device__ __forceinline__ void named_barrier(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

constexpr int kMaxRowWarps = 16;  // warps that share a row
constexpr int kMaxSums = 8;

// ---------------------------------------------------------------------------
// A ring of rows in shared memory.  Every thread copies its own octets of the next rows with
// 16-byte asynchronous copies and reads only those, so that no thread waits for another's;
// the rows in flight hide memory's latency whatever the registers hold.  Stage `s` keeps
// piece k of a thread at (s * pieces + k) * threads + thread.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// Until at most `n` (0 .. 5) of this thread's groups are in flight.
__device__ __forceinline__ void copies_wait(int n) {
  if (n == 0)
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  else if (n == 1)
    asm volatile("cp.async.wait_group 1;" ::: "memory");
  else if (n == 2)
    asm volatile("cp.async.wait_group 2;" ::: "memory");
  else if (n == 3)
    asm volatile("cp.async.wait_group 3;" ::: "memory");
  else if (n == 4)
    asm volatile("cp.async.wait_group 4;" ::: "memory");
  else
    asm volatile("cp.async.wait_group 5;" ::: "memory");
}
constexpr int kMaxStages = 6;

__device__ __forceinline__ uint4 ld_shared16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

// Octet `o` of a row of T to shared memory, its 16-byte pieces `step` apart; and back.
template <class T>
__device__ __forceinline__ void copy_octet(uint32_t dst, uint32_t step, const void* row, int o) {
  const uint8_t* src = static_cast<const uint8_t*>(row) + o * (8 * Elem<T>::kBytes);
  copy16(dst, src);
  if (Elem<T>::kBytes == 4) copy16(dst + step, src + 16);
}
__device__ __forceinline__ void shared_octet(bf16_t, uint32_t a, uint32_t, float (&f)[8]) {
  octet_floats(ld_shared16(a), f);
}
__device__ __forceinline__ void shared_octet(float, uint32_t a, uint32_t step, float (&f)[8]) {
  Elem<float>::Octet o;
  o.a = ld_shared16(a);
  o.b = ld_shared16(a + step);
  octet_floats(o, f);
}
template <class T>
constexpr int kPieces = Elem<T>::kBytes / 2;  // 16-byte pieces of an octet

// ---------------------------------------------------------------------------
// Sums over a row that `warps` warps of the CTA share.  Every thread gets them, added in
// an order that does not depend on timing.  Two sets of slots in turn: a warp that writes
// one has passed the barrier that everybody reached after reading it.
struct RowSums {
  float (*slots)[kMaxSums][kMaxRowWarps];  // [2], of this row group; unused warps hold 0
  int warps, warp, id;                     // of the group; barrier 1 + id
  uint32_t turn;

  // The largest of values that are not negative.
  __device__ __forceinline__ float max(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
    if (warps == 1) return v;
    float* s = slots[turn & 1][0];
    ++turn;
    if ((threadIdx.x & 31) == 0) s[warp] = v;
    named_barrier(1 + id, warps * 32);
    for (int w = 0; w < warps; ++w) v = fmaxf(v, s[w]);
    return v;
  }

  // K sums (1, 2, 4 or 8) at once.  In a warp, each of the first log2 K exchanges also
  // halves the number of sums that a lane goes on with, so that K sums take K + 4 - log2 K
  // exchanges and lane l ends with sum l / (32 / K); the warps' sums are read back in the
  // same arrangement.
  template <int K>
  __device__ __forceinline__ void add(float (&v)[K]) {
    static_assert(K == 1 || K == 2 || K == 4 || K == 8, "a power of two");
    constexpr int kLanes = 32 / K;  // that hold the same sum
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int n = K / 2, d = 16; n > 0; n >>= 1, d >>= 1) {
      const bool up = lane & d;
#pragma unroll
      for (int k = 0; k < n; ++k) {
        const float give = up ? v[k] : v[k + n];
        v[k] = (up ? v[k + n] : v[k]) + __shfl_xor_sync(0xffffffffu, give, d);
      }
    }
#pragma unroll
    for (int d = kLanes / 2; d > 0; d >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], d);
    float t = v[0];
    if (warps > 1) {
      float(*s)[kMaxRowWarps] = slots[turn & 1];
      ++turn;
      const int k = lane / kLanes;
      if (lane % kLanes == 0) s[k][warp] = t;
      named_barrier(1 + id, warps * 32);
      if (K == 8) {
        const float4 q = *reinterpret_cast<const float4*>(&s[k][4 * (lane & 3)]);
        t = (q.x + q.y) + (q.z + q.w);
      } else if (K == 4) {
        const float2 q = *reinterpret_cast<const float2*>(&s[k][2 * (lane & 7)]);
        t = q.x + q.y;
      } else {
        t = s[k][lane & 15];
      }
      constexpr int kHold = K == 1 ? 16 : kLanes;  // lanes that share a sum's parts
#pragma unroll
      for (int d = kHold / 2; d > 0; d >>= 1) t += __shfl_xor_sync(0xffffffffu, t, d);
    }
    if (K == 1) {
      v[0] = t;
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] = __shfl_sync(0xffffffffu, t, k * kLanes);
    }
  }
};

}  // namespace flce
