// Microscaled 4-bit blocks (include/gptq_mx.h): 32 elements sharing a scale 2^(e-127),
// each a code sign << 3 | magnitude with magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6; and the
// loads and stores that the row quantiser and the cache share.
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
__device__ __forceinline__ uint32_t encode8(const float* v) {
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

// The levels of the 4 or 8 lowest codes of w (exact in fp16).
template <int N>
__device__ __forceinline__ void decode(uint32_t w, float (&v)[N]) {
  static_assert(N == 4 || N == 8, "codes of half a word or a word");
  uint32_t h[4] = {0, 0, 0, 0};
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t}"
      : "=r"(h[0]), "=r"(h[1])
      : "r"(w));
  if (N == 8)
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, d;\n\t}"
        : "=r"(h[2]), "=r"(h[3])
        : "r"(w));
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

// The values of eight codes in fp16, for scales 2^-24 .. 2^15 (103 <= e <= 142).
__device__ __forceinline__ uint4 decode8_half(uint32_t w, uint32_t e) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
  const __half2 f = __float2half2_rn(__uint_as_float(e << 23));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 p = __hmul2(*reinterpret_cast<const __half2*>(&h[i]), f);
    h[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(h[0], h[1], h[2], h[3]);
}

// Byte offset of the scale of (row, block) in 128 x 4 tiles, `ct` tiles per tile row.
__device__ __forceinline__ int64_t scale_offset(int64_t row, int block, int ct) {
  return ((row >> 7) * ct + (block >> 2)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 +
         (block & 3);
}

}  // namespace mx

template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32(float x) { return x; }
template <> __device__ __forceinline__ __half from_f32(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32(float x) { return __float2bfloat16_rn(x); }

// min and max that return NaN if either side is one
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// 32 bytes of a row in one lane, as loaded: 8 fp32 or 16 16-bit elements.  A warp's two 16-byte
// loads then use whole 32-byte sectors, and the per-lane work of a group (its range, its grid,
// its addresses) is shared by twice the 16-bit elements of a 16-byte unit.
template <typename T>
struct Unit {
  static constexpr int N = 32 / int(sizeof(T));
  static constexpr int WORDS = N / 8;          // words of 4-bit codes
  uint4 q[2];

  // `n` elements exist (more than N: all; the others read as 0); vec: p is a multiple of 16 bytes
  __device__ __forceinline__ void load(const T* p, int n, bool vec) {
    q[0] = q[1] = make_uint4(0u, 0u, 0u, 0u);
    if (vec && n >= N / 2) {
      q[0] = *reinterpret_cast<const uint4*>(p);
      if (n >= N) q[1] = reinterpret_cast<const uint4*>(p)[1];
      else set_some(p, N / 2, n);
    } else {
      set_some(p, 0, n);
    }
  }
  __device__ __forceinline__ void set_some(const T* p, int from, int n) {
    __align__(16) T e[N];
    *reinterpret_cast<uint4*>(e) = q[0];
    *reinterpret_cast<uint4*>(e + N / 2) = q[1];
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i >= from && i < n) e[i] = p[i];
    q[0] = *reinterpret_cast<uint4*>(e);
    q[1] = *reinterpret_cast<uint4*>(e + N / 2);
  }
  // The same from any address: where the three 16-byte granules that hold the unit lie inside
  // [lo, hi) they are loaded whole (begin) and the unit's bytes shifted out of them (finish).
  __device__ __forceinline__ bool begin(const T* p, int n, const T* lo, const T* hi, uint4& q2) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p) & ~uintptr_t(15);
    const bool whole = n >= N && at >= reinterpret_cast<uintptr_t>(lo) &&
                       at + 48 <= reinterpret_cast<uintptr_t>(hi);
    q2 = make_uint4(0u, 0u, 0u, 0u);
    if (whole) {
      const uint4* g = reinterpret_cast<const uint4*>(at);
      q[0] = g[0];
      q[1] = g[1];
      q2 = g[2];
    } else {
      q[0] = q[1] = q2;
      set_some(p, 0, n);
    }
    return whole;
  }
  __device__ __forceinline__ void finish(const T* p, bool whole, const uint4& q2) {
    const uint32_t off = whole ? uint32_t(reinterpret_cast<uintptr_t>(p)) & 15u : 0u;
    uint32_t w[12] = {q[0].x, q[0].y, q[0].z, q[0].w, q[1].x, q[1].y, q[1].z, q[1].w,
                      q2.x, q2.y, q2.z, q2.w};
    shift_words<12>(w, off);
    q[0] = make_uint4(w[0], w[1], w[2], w[3]);
    q[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
  // w = w shifted down by off < 16 bytes (a multiple of the element size)
  template <int W>
  static __device__ __forceinline__ void shift_words(uint32_t (&w)[W], uint32_t off) {
#pragma unroll
    for (int i = 0; i + 1 < W; ++i) w[i] = off & 4 ? w[i + 1] : w[i];
#pragma unroll
    for (int i = 0; i + 2 < W; ++i) w[i] = off & 8 ? w[i + 2] : w[i];
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i + 1 < W; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 8 * (off & 3));
    }
  }
  __device__ __forceinline__ uint32_t word(int i) const {
    const uint4& a = q[i >> 2];
    return (i & 3) == 0 ? a.x : (i & 3) == 1 ? a.y : (i & 3) == 2 ? a.z : a.w;
  }
  __device__ __forceinline__ void widen(float (&v)[N]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t w = word(i);
      if constexpr (sizeof(T) == 4) {
        v[i] = __uint_as_float(w);
      } else if constexpr (__is_same(T, __half)) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      } else {
        v[2 * i] = __uint_as_float(w << 16);
        v[2 * i + 1] = __uint_as_float(w & 0xFFFF0000u);
      }
    }
  }
  // fp32 bits of the largest magnitude (a NaN's or an infinity's are above the finite ones')
  __device__ __forceinline__ uint32_t amax_bits() const {
    constexpr uint32_t mag = sizeof(T) == 4 ? 0x7FFFFFFFu : 0x7FFF7FFFu;
    uint32_t m = word(0) & mag;
#pragma unroll
    for (int i = 1; i < 8; ++i) {
      if constexpr (sizeof(T) == 4) m = max(m, word(i) & mag);
      else m = __vmaxu2(m, word(i) & mag);
    }
    if constexpr (sizeof(T) == 4) return m;
    m = max(m & 0xFFFFu, m >> 16);
    if constexpr (__is_same(T, __half)) return __float_as_uint(__half2float(__ushort_as_half(uint16_t(m))));
    return m << 16;
  }
  // smallest and largest value; NaN if any is
  __device__ __forceinline__ void range(float& lo, float& hi) const {
    if constexpr (sizeof(T) == 4) {
      lo = hi = __uint_as_float(word(0));
#pragma unroll
      for (int i = 1; i < 8; ++i) {
        lo = min_nan(lo, __uint_as_float(word(i)));
        hi = max_nan(hi, __uint_as_float(word(i)));
      }
    } else if constexpr (__is_same(T, __half)) {
      const auto at = [&](int i) { const uint32_t w = word(i); return *reinterpret_cast<const __half2*>(&w); };
      __half2 a = at(0), b = a;
#pragma unroll
      for (int i = 1; i < 8; ++i) { a = __hmin2_nan(a, at(i)); b = __hmax2_nan(b, at(i)); }
      const float2 fa = __half22float2(a), fb = __half22float2(b);
      lo = min_nan(fa.x, fa.y);
      hi = max_nan(fb.x, fb.y);
    } else {
      const auto at = [&](int i) { const uint32_t w = word(i); return *reinterpret_cast<const __nv_bfloat162*>(&w); };
      __nv_bfloat162 a = at(0), b = a;
#pragma unroll
      for (int i = 1; i < 8; ++i) { a = __hmin2_nan(a, at(i)); b = __hmax2_nan(b, at(i)); }
      lo = min_nan(__low2float(a), __high2float(a));
      hi = max_nan(__low2float(b), __high2float(b));
    }
  }
};

// 16 bytes of a row written by one lane, neighbouring lanes side by side: N = 4 fp32 or 8 16-bit
// elements.
template <typename T>
struct Out {
  static constexpr int N = 16 / int(sizeof(T));
  static __device__ __forceinline__ uint4 pack(const float (&v)[N]) {
    if constexpr (sizeof(T) == 4) {
      return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                        __float_as_uint(v[3]));
    } else {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (__is_same(T, __half)) {
          const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
          w[i] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
          const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
          w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
      }
      return make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  // Elements from .. n-1 of the unit: the whole of it at once, which p's 16 bytes must be
  // aligned for, or one by one.
  static __device__ __forceinline__ void store_some(T* p, int from, int n, const float (&v)[N]) {
    if (from <= 0 && n >= N) {
      *reinterpret_cast<uint4*>(p) = pack(v);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i >= from && i < n) p[i] = from_f32<T>(v[i]);
    }
  }
  // `n` elements exist; vec: p is a multiple of 16 bytes
  static __device__ __forceinline__ void store(T* p, int n, bool vec, const float (&v)[N]) {
    if (vec && n >= N) {
      *reinterpret_cast<uint4*>(p) = pack(v);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i < n) p[i] = from_f32<T>(v[i]);
    }
  }
};

}  // namespace gptq
