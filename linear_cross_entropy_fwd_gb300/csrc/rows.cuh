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

// An octet in fp32, as four pairs: the arithmetic on it is two elements an instruction.
struct Oct {
  float2 p[4];
};

__device__ __forceinline__ float2 pair(float x) { return make_float2(x, x); }

__device__ __forceinline__ float2 pair_op(uint64_t d) { return reinterpret_cast<const float2&>(d); }
__device__ __forceinline__ uint64_t pair_bits(const float2& a) {
  return reinterpret_cast<const uint64_t&>(a);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(pair_bits(a)), "l"(pair_bits(b)));
  return pair_op(d);
}
__device__ __forceinline__ float2 plus2(float2 a, float2 b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(pair_bits(a)), "l"(pair_bits(b)));
  return pair_op(d);
}
__device__ __forceinline__ float2 mad2(float2 a, float2 b, float2 c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(d)
      : "l"(pair_bits(a)), "l"(pair_bits(b)), "l"(pair_bits(c)));
  return pair_op(d);
}

__device__ __forceinline__ Oct zero_oct() {
  Oct o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o.p[i] = pair(0.f);
  return o;
}
__device__ __forceinline__ Oct same_oct(float x) {
  Oct o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o.p[i] = pair(x);
  return o;
}
__device__ __forceinline__ void scale_oct(Oct& x, const Oct& f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) x.p[i] = mul2(x.p[i], f.p[i]);
}
__device__ __forceinline__ void scale_oct(Oct& x, float f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) x.p[i] = mul2(x.p[i], pair(f));
}
__device__ __forceinline__ void add_oct(Oct& x, const Oct& y) {
#pragma unroll
  for (int i = 0; i < 4; ++i) x.p[i] = plus2(x.p[i], y.p[i]);
}
__device__ __forceinline__ float sum_oct(const Oct& x) {
  const float2 t = plus2(plus2(x.p[0], x.p[1]), plus2(x.p[2], x.p[3]));
  return t.x + t.y;
}

__device__ __forceinline__ Oct from_octet(const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  Oct o;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o.p[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  return o;
}
__device__ __forceinline__ Oct from_octet(const Elem<float>::Octet& v) {
  Oct o;
  o.p[0] = make_float2(__uint_as_float(v.a.x), __uint_as_float(v.a.y));
  o.p[1] = make_float2(__uint_as_float(v.a.z), __uint_as_float(v.a.w));
  o.p[2] = make_float2(__uint_as_float(v.b.x), __uint_as_float(v.b.y));
  o.p[3] = make_float2(__uint_as_float(v.b.z), __uint_as_float(v.b.w));
  return o;
}

__device__ __forceinline__ uint4 to_octet(bf16_t, const Oct& f) {
  return make_uint4(pack_bf16x2(f.p[0].x, f.p[0].y), pack_bf16x2(f.p[1].x, f.p[1].y),
                    pack_bf16x2(f.p[2].x, f.p[2].y), pack_bf16x2(f.p[3].x, f.p[3].y));
}
__device__ __forceinline__ Elem<float>::Octet to_octet(float, const Oct& f) {
  Elem<float>::Octet o;
  o.a = make_uint4(__float_as_uint(f.p[0].x), __float_as_uint(f.p[0].y),
                   __float_as_uint(f.p[1].x), __float_as_uint(f.p[1].y));
  o.b = make_uint4(__float_as_uint(f.p[2].x), __float_as_uint(f.p[2].y),
                   __float_as_uint(f.p[3].x), __float_as_uint(f.p[3].y));
  return o;
}

// Octet `o` of a row of T at `row`.
template <class T>
__device__ __forceinline__ Oct load_octet(const void* row, int o) {
  return from_octet(static_cast<const typename Elem<T>::Octet*>(row)[o]);
}
template <class T>
__device__ __forceinline__ void store_octet(void* row, int o, const Oct& f) {
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
__device__ __forceinline__ Oct param_octet(const void* p, bool fp32, int o, float missing) {
  if (!p) return same_oct(missing);
  return fp32 ? load_octet<float>(p, o) : load_octet<T>(p, o);
}

// One element of type T, or fp32: its bits, for a load that nothing waits for yet, and its value.
template <class T>
__device__ __forceinline__ uint32_t element_bits(const void* p, bool fp32, int64_t i) {
  if (fp32 || Elem<T>::kBytes == 4) return static_cast<const uint32_t*>(p)[i];
  return static_cast<const uint16_t*>(p)[i];
}
template <class T>
__device__ __forceinline__ float element_value(uint32_t bits, bool fp32) {
  return __uint_as_float(fp32 || Elem<T>::kBytes == 4 ? bits : bits << 16);
}
template <class T>
__device__ __forceinline__ float one_element(const void* p, bool fp32, int64_t i) {
  return element_value<T>(element_bits<T>(p, fp32, i), fp32);
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
// A ring of rows in shared memory.  Every warp copies its own octets of the next rows with
// 16-byte asynchronous copies and reads only those, so that no warp waits for another's;
// the rows in flight hide memory's latency whatever the registers hold.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// Until at most N of this thread's groups are in flight.
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Stages of a ring whose threads keep `pieces` pieces in each.
constexpr int ring_stages(int pieces, int threads, int bytes, int most) {
  return bytes / (pieces * threads * 16) < most ? bytes / (pieces * threads * 16) : most;
}

__device__ __forceinline__ void st_shared4(uint32_t a, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_shared4(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

// A thread's place for one octet of T in each stage.  A bf16 octet is one 16-byte piece.  An
// fp32 octet is two: a warp's 32 octets are copied as 64 pieces side by side (each lane's
// two pieces next to one another would ask for every 32-byte sector twice), so lanes read
// what others copied, after a __syncwarp.  Piece c lies at c ^ (c >> 3 & 1), which spreads a
// quarter warp's reads of every other piece over all banks.
template <class T>
struct Slot;
template <>
struct Slot<bf16_t> {
  uint32_t at;
  bool there;
  __device__ __forceinline__ Slot(int thread, int, int octet, int octets)
      : at(thread * 16), there(octet < octets) {}
  static constexpr bool kOwn = true;  // a lane copies what it reads
  __device__ __forceinline__ void copy(uint32_t region, const uint8_t* octet, bool known) const {
    if (known || there) copy16(region + at, octet);
  }
  __device__ __forceinline__ Oct read(uint32_t region) const {
    return from_octet(ld_shared16(region + at));
  }
};
template <>
struct Slot<float> {
  uint32_t to, first, second;
  int back;
  bool a, b;
  __device__ __forceinline__ Slot(int thread, int lane, int octet, int octets)
      : back(16 * lane),
        a(octet - lane + lane / 2 < octets),
        b(octet - lane + 16 + lane / 2 < octets) {
    const uint32_t warp = (thread - lane) * 32, flip = lane >> 2 & 1;
    to = warp + (lane ^ (lane >> 3 & 1)) * 16;
    first = warp + ((2 * lane) ^ flip) * 16;
    second = warp + ((2 * lane + 1) ^ flip) * 16;
  }
  static constexpr bool kOwn = false;
  __device__ __forceinline__ void copy(uint32_t region, const uint8_t* octet, bool) const {
    if (a) copy16(region + to, octet - back);
    if (b) copy16(region + to + 512, octet - back + 512);
  }
  __device__ __forceinline__ Oct read(uint32_t region) const {
    Elem<float>::Octet o;
    o.a = ld_shared16(region + first);
    o.b = ld_shared16(region + second);
    return from_octet(o);
  }
};

// An fp32 octet kept as two planes `step` bytes apart.
__device__ __forceinline__ Oct shared_oct(uint32_t a, uint32_t step) {
  Elem<float>::Octet o;
  o.a = ld_shared16(a);
  o.b = ld_shared16(a + step);
  return from_octet(o);
}

__device__ __forceinline__ void put_octet(void* at, const uint4& o, bool) {
  *static_cast<uint4*>(at) = o;
}
// `wide`: 32-byte aligned, so that a store covers whole sectors.
__device__ __forceinline__ void put_octet(void* at, const Elem<float>::Octet& o, bool wide) {
  if (wide)
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(o.a.x),
                 "r"(o.a.y), "r"(o.a.z), "r"(o.a.w), "r"(o.b.x), "r"(o.b.y), "r"(o.b.z),
                 "r"(o.b.w)
                 : "memory");
  else
    *static_cast<Elem<float>::Octet*>(at) = o;
}

// A thread's octet of one row after the other.  The step to the next one is a launch
// parameter, so that it takes no registers.
template <class T>
struct Walk {
  uint8_t* at;
  __device__ __forceinline__ Walk(const void* base, int64_t row_stride, int64_t row, int octet)
      : at(static_cast<uint8_t*>(const_cast<void*>(base)) +
           (row * row_stride + 8 * octet) * Elem<T>::kBytes) {}
  __device__ __forceinline__ void put(const typename Elem<T>::Octet& o, bool wide,
                                      int64_t bytes = 0) const {
    put_octet(at + bytes, o, wide);
  }
};
__device__ __forceinline__ void put_shared(uint32_t a, uint32_t step, const Oct& o) {
  const Elem<float>::Octet v = to_octet(float{}, o);
  st_shared_v4(a, v.a.x, v.a.y, v.a.z, v.a.w);
  st_shared_v4(a + step, v.b.x, v.b.y, v.b.z, v.b.w);
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
      if (K == 1) {  // fewer steps one after the other than exchanges would take
        const float4 q = *reinterpret_cast<const float4*>(&s[0][0]);
        t = (q.x + q.y) + (q.z + q.w);
        for (int w = 4; w < warps; w += 4) {
          const float4 r = *reinterpret_cast<const float4*>(&s[0][w]);
          t += (r.x + r.y) + (r.z + r.w);
        }
        v[0] = t;
        return;
      }
      if (K == 8) {
        const float4 q = *reinterpret_cast<const float4*>(&s[k][4 * (lane & 3)]);
        t = (q.x + q.y) + (q.z + q.w);
      } else if (K == 4) {
        const float2 q = *reinterpret_cast<const float2*>(&s[k][2 * (lane & 7)]);
        t = q.x + q.y;
      } else {
        t = s[k][lane & 15];
      }
#pragma unroll
      for (int d = kLanes / 2; d > 0; d >>= 1) t += __shfl_xor_sync(0xffffffffu, t, d);
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
