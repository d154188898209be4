// ckpt.cuh -- the format of an 8-bit activation checkpoint.
//
// 32 consecutive values of a row share a scale 2^e, e the smallest with |v| <= 448 2^e for
// all of them (448 is e4m3's largest number), within -117 .. 119.  A power of two, so that
// a stored value has 4 significant bits and is exact in bf16: the weight gradient's products
// are those of the stored values, with no second rounding.  The bounds keep the smallest
// stored value, 2^(e - 9), a normal number and the largest finite.  A scale byte of 255
// marks a group with a NaN or an infinity, which comes back as NaN.
#pragma once
#include "rows.cuh"

namespace flce {

struct Ckpt {
  uint8_t* codes;   // [N][pitch]
  uint8_t* scales;  // [N][spitch], e + 127
  int32_t pitch, spitch;
};

inline __host__ __device__ int32_t ckpt_pitch(int64_t H) {
  return static_cast<int32_t>((H + 31) / 32 * 32);
}
inline __host__ __device__ int32_t ckpt_spitch(int64_t H) {
  return static_cast<int32_t>((H + 127) / 128 * 4);
}
inline Ckpt ckpt_view(void* p, int64_t N, int64_t H) {
  Ckpt c;
  c.pitch = ckpt_pitch(H);
  c.spitch = ckpt_spitch(H);
  c.codes = static_cast<uint8_t*>(p);
  c.scales = c.codes + N * c.pitch;
  return c;
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(lo), "f"(hi));
  return r;
}

__device__ __forceinline__ float2 from_e4m3x2(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(codes)));
  float2 f;
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\t"
      "cvt.f32.f16 %1, b;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}

// The bits of the largest magnitude of an octet, as fp32; NaN above infinity's.
__device__ __forceinline__ uint32_t octet_top(const uint4& v) {
  uint32_t m = v.x & 0x7fff7fffu;
  const uint32_t w[3] = {v.y & 0x7fff7fffu, v.z & 0x7fff7fffu, v.w & 0x7fff7fffu};
#pragma unroll
  for (int i = 0; i < 3; ++i) asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i]));
  return max(m << 16, m & 0x7fff0000u);
}
__device__ __forceinline__ uint32_t octet_top(const Elem<float>::Octet& v) {
  const uint32_t w[8] = {v.a.x, v.a.y, v.a.z, v.a.w, v.b.x, v.b.y, v.b.z, v.b.w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, w[i] & 0x7fffffffu);
  return m;
}

// Stores octet `o` of a row whose octet goes to `codes` and whose scales begin at `scales`:
// v holds its values (zeros behind the row's end, where `o` may lie too).  Executed by whole
// warps whose lanes hold consecutive octets, lane 0 a multiple of 4, so that four lanes hold
// a group.
template <class OctetT>
__device__ __forceinline__ void ckpt_store_octet(const Ckpt& c, uint8_t* codes, uint8_t* scales,
                                                 int o, const OctetT& v) {
  uint32_t top = octet_top(v);
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  // ceil(log2(top / 448)) + 127: 448 = 1.75 * 2^8, and a mantissa above .75 carries
  int s = static_cast<int>((top + 0x1fffffu) >> 23) - 8;
  s = min(max(s, 127 - 117), 127 + 119);
  const float2 inv = pair(__uint_as_float(static_cast<uint32_t>(254 - s) << 23));  // 2^-e
  const Oct x = from_octet(v);
  uint32_t q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = mul2(x.p[i], inv);
    q[i] = e4m3x2(t.x, t.y);
  }
  uint2 w = make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
  if (top >= 0x7f800000u) {
    s = 255;
    w = make_uint2(0, 0);
  }
  if (o * 8 >= c.pitch) return;
  *reinterpret_cast<uint2*>(codes) = w;
  if ((o & 3) == 0) {
    int g = o >> 2;
    scales[g] = static_cast<uint8_t>(s);
    if (o * 8 + 32 == c.pitch)
      while (++g < c.spitch) scales[g] = 0;
  }
}

// 2^e of a scale byte, NaN for 255.
__device__ __forceinline__ float ckpt_scale(uint32_t byte) {
  return __uint_as_float(byte == 255 ? 0x7fffffffu : byte << 23);
}

// The octet of these codes and this scale byte.
__device__ __forceinline__ Oct ckpt_octet(const uint2& codes, uint32_t scale) {
  const float f = ckpt_scale(scale);
  Oct x;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    x.p[i] = mul2(from_e4m3x2((i < 2 ? codes.x : codes.y) >> (16 * (i & 1))), pair(f));
  return x;
}

// x [N, H] = the checkpoint; elements of 2 (bf16) or 4 bytes, rows x_row elements apart.
// `clear`, if not null, becomes 0, and the next launch may start meanwhile.
cudaError_t launch_ckpt_load(const Ckpt& c, void* x, int64_t x_row, int64_t N, int64_t H, int elt,
                             int32_t* clear, cudaStream_t s);

}  // namespace flce
