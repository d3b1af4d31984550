// Microscaled 4-bit blocks (include/gptq_mx.h): 32 elements sharing a scale 2^(e-127),
// each a code sign << 3 | magnitude with magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6.  Shared by
// the row quantiser and the cache.  Lanes work on units of 8 consecutive elements, the
// eight codes of one 32-bit word, so a block is 4 neighbouring lanes.
#pragma once
#include "common.cuh"

namespace gptq {
namespace mx {

// Scale byte of a block from the bits of its largest magnitude (fp32, sign cleared; a NaN's
// or an infinity's bits are above every finite value's): the largest magnitude's biased
// exponent less 2, the exponent of the largest level, 4 <= 6 < 8; 255 if it is not finite.
__device__ __forceinline__ int scale_byte(uint32_t amax_bits) {
  const int E = int(amax_bits >> 23);
  return E == 255 ? 255 : max(E - 2, 0);
}

// 2^(127 - e) for e <= 253: exact, so that x * inv_scale is x / 2^(e-127) (a result below
// fp32's normal range may round, but every such result is far below 0.25 and becomes 0)
__device__ __forceinline__ float inv_scale(int e) { return __uint_as_float(uint32_t(254 - e) << 23); }

// 2^(e-127); e = 0 is an fp32 subnormal, e = 255 not a number
__device__ __forceinline__ float scale_value(uint32_t e) {
  return __uint_as_float(e == 0u ? 0x00400000u : e == 255u ? 0x7FC00000u : e << 23);
}

// Eight values, already divided by the scale, to eight codes (round to nearest, ties to the
// even code, saturating): the first value in the lowest bits.
__device__ __forceinline__ uint32_t encode8(const float (&v)[8]) {
  uint32_t w;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(w)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return w;
}

// The levels of eight codes (exact in fp16).
__device__ __forceinline__ void decode8(uint32_t w, float (&v)[8]) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

// Bits of the largest magnitude of eight values.
__device__ __forceinline__ uint32_t amax_bits8(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  return m;
}

// Byte offset of the scale of (row, block) in 128 x 4 tiles, `ct` tiles per tile row.
__device__ __forceinline__ int64_t scale_offset(int64_t row, int block, int ct) {
  return ((row >> 7) * ct + (block >> 2)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 +
         (block & 3);
}

}  // namespace mx

template <typename T>
__device__ __forceinline__ float to_f32(T x);
template <> __device__ __forceinline__ float to_f32(float x) { return x; }
template <> __device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
template <> __device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32(float x) { return x; }
template <> __device__ __forceinline__ __half from_f32(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32(float x) { return __float2bfloat16_rn(x); }

// A unit's raw bits as loaded (16 or 32 bytes), so that several loads can be in flight
// before the first is used.
template <typename T>
struct Raw8 {
  union {
    uint4 q[sizeof(T) / 2];
    T e[8];
  };
  __device__ Raw8() {}
};

// Eight consecutive elements, of which `n` exist (the others read as 0); `vec`: the address
// is a multiple of 16 bytes.
template <typename T>
__device__ __forceinline__ void load8(const T* p, int n, bool vec, Raw8<T>& r) {
  if (vec && n >= 8) {
#pragma unroll
    for (int i = 0; i < int(sizeof(T)) / 2; ++i) r.q[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.e[i] = i < n ? p[i] : from_f32<T>(0.f);
  }
}

template <typename T>
__device__ __forceinline__ void widen8(const Raw8<T>& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = to_f32<T>(r.e[i]);
}

template <typename T>
__device__ __forceinline__ void store8(T* p, int n, bool vec, const float (&v)[8]) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < 8; ++i) r.e[i] = from_f32<T>(v[i]);
  if (vec && n >= 8) {
#pragma unroll
    for (int i = 0; i < int(sizeof(T)) / 2; ++i) reinterpret_cast<uint4*>(p)[i] = r.q[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = r.e[i];
  }
}

}  // namespace gptq
