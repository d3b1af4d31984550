// The paged low-bit key/value cache (include/gptq_cache.h): rows are quantised as they are
// written and read back as floating point.
//
// Both directions are one pass over the rows, bound by HBM (2 or 4 bytes per value on one
// side, 4.25 to 10 bits on the other) or, for a token per sequence, by the launch and the
// chain cu -> start -> table -> slot.  A lane holds a unit of 8 values (16 or 32 bytes of a
// row, one or two words of codes) and a group is 1 to 32 neighbouring lanes, so a group's
// range is a few shuffles and nothing is staged.  A CTA takes a few consecutive rows; one
// thread per row finds its sequence and slot while the other threads' loads are in flight.
#include <algorithm>

#include "grid.cuh"
#include "kernels.h"
#include "kv_slots.h"
#include "mx.cuh"

namespace gptq {
namespace {

constexpr int THREADS = 256;
constexpr int STEPS = 4;          // units of a thread whose loads are issued together
constexpr int MAX_ROWS = 64;      // rows of a CTA

// n / d for 0 <= n < 2^31 by a multiplication: with 2^(s-1) < d <= 2^s and
// m = ceil(2^(31+s) / d), m / 2^(31+s) exceeds 1/d by less than 2^-(31+s), so the product
// with n < 2^31 exceeds n / d by less than 2^-s <= 1/d, too little to reach the next whole number.
struct Div {
  uint32_t d, m, s;
  explicit Div(uint32_t d_) : d(d_), m(0), s(0) {
    while ((1ull << s) < d) ++s;
    m = uint32_t(((1ull << (31 + s)) + d - 1) / d);
  }
  __device__ __forceinline__ uint32_t quot(uint32_t n) const {
    return uint32_t((uint64_t(n) * m) >> (31 + s));
  }
};

struct Args {
  const void* in[2];     // write: K and V
  void* out[2];          // read: K and V
  int64_t ldt[2], ldh[2];
  uint32_t* codes[2];
  void* grids[2];
  RowMap map;
  int64_t tokens;
  int heads, units, words, groups;   // units of 8 values, words and groups of one head
  int lane_bits;                     // a group is 2^lane_bits lanes
  int rows;                          // rows of a CTA
  int vec;                           // all rows on 16-byte boundaries
  int sym;
  Div per_row, per_kv, per_head;     // lanes of a row (K and V), of K alone, of a head
};

// The slot of row t, negative if it has none.
__device__ __forceinline__ int64_t find_slot(const Args& a, int64_t t, int32_t* status) {
  const int64_t slot = slot_of(a.map, t);
  if (slot == SLOT_BAD) raise_status(status, GPTQ_ERR_INVALID_ARG);
  return slot;
}

// What a thread's lane of a CTA works on: row (in the CTA), K or V, head, group, unit.
struct Place {
  int row, kv, head, group, unit;
  bool live;       // the unit holds words of the stored form
};

__device__ __forceinline__ Place place_of(const Args& a, uint32_t i) {
  Place p;
  p.row = int(a.per_row.quot(i));
  i -= uint32_t(p.row) * a.per_row.d;
  p.kv = i >= a.per_kv.d;
  i -= p.kv ? a.per_kv.d : 0u;
  p.head = int(a.per_head.quot(i));
  i -= uint32_t(p.head) * a.per_head.d;
  p.group = int(i) >> a.lane_bits;
  p.unit = int(i);
  return p;
}

enum { GRID4 = 0, GRID8 = 1, MX4 = 2 };

// rint(x / s) with the quotient rounded to fp32: the product with 1/s is within 2^-15 of it
// for |x / s| <= 256, so only a product that near a half-integer needs the division.
__device__ __forceinline__ float rint_quot(float x, float s, float inv, bool divide) {
  const float q = x * inv, r = rintf(q);
  if (divide || fabsf(q - r) > 0.49995f) return rintf(__fdiv_rn(x, s));
  return r;
}

template <typename T, int KIND>
__global__ void __launch_bounds__(THREADS)
k_cache_write(const Args a, int32_t* status) {
  __shared__ int64_t slots[MAX_ROWS];
  const int64_t t0 = int64_t(blockIdx.x) * a.rows;
  const int rows = int(min(int64_t(a.rows), a.tokens - t0));
  const uint32_t total = uint32_t(rows) * a.per_row.d;
  bool bad = false, ready = false;
  for (uint32_t i0 = threadIdx.x; i0 - threadIdx.x < total; i0 += THREADS * STEPS) {
    Raw8<T> raw[STEPS];
    Place pl[STEPS];
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const uint32_t i = i0 + s * THREADS;
      pl[s] = place_of(a, i);
      const int n = i < total ? (a.units - pl[s].unit) * 8 : 0;
      const T* p = static_cast<const T*>(a.in[pl[s].kv]) + (t0 + pl[s].row) * a.ldt[pl[s].kv] +
                   pl[s].head * a.ldh[pl[s].kv] + pl[s].unit * 8;
      load8(p, n, a.vec != 0, raw[s]);
    }
    if (!ready) {
      if (int(threadIdx.x) < rows) slots[threadIdx.x] = find_slot(a, t0 + threadIdx.x, status);
      __syncthreads();
      ready = true;
    }
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const bool in = i0 + s * THREADS < total;
      const int64_t slot = in ? slots[pl[s].row] : -1;
      float v[8];
      widen8(raw[s], v);
      const int64_t head = slot * a.heads + pl[s].head;
      uint32_t* codes = a.codes[pl[s].kv] + head * a.words;
      uint32_t m = mx::amax_bits8(v);
      if constexpr (KIND == MX4) {
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const int e = mx::scale_byte(m);
        uint32_t w = 0;
        if (e != 255) {
          const float f = mx::inv_scale(e);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] *= f;
          w = mx::encode8(v);
        }
        if (slot >= 0) {
          bad |= e == 255;
          codes[pl[s].unit] = w;
          if ((pl[s].unit & 3) == 0)
            static_cast<uint8_t*>(a.grids[pl[s].kv])[head * a.groups + pl[s].group] = uint8_t(e);
        }
      } else {
        constexpr float maxq = KIND == GRID4 ? 15.f : 255.f;
        float lo = 0.f, hi = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) { lo = fminf(lo, v[j]); hi = fmaxf(hi, v[j]); }
        for (int o = 1; o < (1 << a.lane_bits); o <<= 1) {
          m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
          lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
          hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        }
        float sc, z;
        grid_params(lo, hi, maxq, a.sym, sc, z);
        if (sc == 0.f) grid_params(-1.f, 1.f, maxq, a.sym, sc, z);   // an underflowed range
        const bool nan = m >= 0x7F800000u || __float_as_uint(sc) >= 0x7F800000u;
        uint32_t w[2] = {0u, 0u};
        if (nan) {
          sc = __uint_as_float(0x7FC00000u);
          z = 0.f;
        } else {
          const bool divide = sc < 0x1p-100f || sc > 0x1p100f;
          const float inv = __frcp_rn(sc);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float c = fminf(fmaxf(rint_quot(v[j], sc, inv, divide) + z, 0.f), maxq);
            if constexpr (KIND == GRID4) w[0] |= uint32_t(c) << (4 * j);
            else w[j >> 2] |= uint32_t(c) << (8 * (j & 3));
          }
        }
        if (slot >= 0 && pl[s].unit < a.units) {
          bad |= nan;
          if constexpr (KIND == GRID4) codes[pl[s].unit] = w[0];
          else *reinterpret_cast<uint2*>(codes + 2 * pl[s].unit) = make_uint2(w[0], w[1]);
          if (pl[s].unit == pl[s].group << a.lane_bits)
            static_cast<float2*>(a.grids[pl[s].kv])[head * a.groups + pl[s].group] = make_float2(sc, z);
        }
      }
    }
  }
  if (bad) raise_status(status, GPTQ_ERR_NONFINITE);
}

template <typename T, int KIND>
__global__ void __launch_bounds__(THREADS)
k_cache_read(const Args a, int32_t* status) {
  __shared__ int64_t slots[MAX_ROWS];
  const int64_t t0 = int64_t(blockIdx.x) * a.rows;
  const int rows = int(min(int64_t(a.rows), a.tokens - t0));
  const uint32_t total = uint32_t(rows) * a.per_row.d;
  if (int(threadIdx.x) < rows) slots[threadIdx.x] = find_slot(a, t0 + threadIdx.x, status);
  __syncthreads();
  for (uint32_t i0 = threadIdx.x; i0 < total; i0 += THREADS * STEPS) {
    uint32_t w[STEPS][2];
    float sc[STEPS], z[STEPS];
    Place pl[STEPS];
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const uint32_t i = i0 + s * THREADS;
      pl[s] = place_of(a, i);
      const int64_t slot = i < total ? slots[pl[s].row] : -1;
      pl[s].live = slot >= 0 && pl[s].unit < a.units;
      if (!pl[s].live) continue;
      const int64_t head = slot * a.heads + pl[s].head;
      const uint32_t* codes = a.codes[pl[s].kv] + head * a.words;
      if constexpr (KIND == GRID8) {
        const uint2 q = __ldg(reinterpret_cast<const uint2*>(codes + 2 * pl[s].unit));
        w[s][0] = q.x;
        w[s][1] = q.y;
      } else {
        w[s][0] = __ldg(codes + pl[s].unit);
      }
      if constexpr (KIND == MX4) {
        sc[s] = mx::scale_value(
            __ldg(static_cast<const uint8_t*>(a.grids[pl[s].kv]) + head * a.groups + pl[s].group));
      } else {
        const float2 g = __ldg(static_cast<const float2*>(a.grids[pl[s].kv]) + head * a.groups + pl[s].group);
        sc[s] = g.x;
        z[s] = g.y;
      }
    }
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      if (!pl[s].live) continue;
      float v[8];
      if constexpr (KIND == MX4) {
        mx::decode8(w[s][0], v);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= sc[s];
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t c = KIND == GRID4 ? (w[s][0] >> (4 * j)) & 15u : (w[s][j >> 2] >> (8 * (j & 3))) & 255u;
          // the code as a float without a conversion: 2^23 + c, less 2^23 (exact)
          v[j] = sc[s] * ((__uint_as_float(0x4B000000u | c) - 8388608.f) - z[s]);
        }
      }
      T* p = static_cast<T*>(a.out[pl[s].kv]) + (t0 + pl[s].row) * a.ldt[pl[s].kv] +
             pl[s].head * a.ldh[pl[s].kv] + pl[s].unit * 8;
      store8(p, 8, a.vec != 0, v);
    }
  }
}

template <typename T, int KIND>
gptq_status launch(cudaStream_t st, bool write, const Args& a, unsigned blocks, int32_t* status) {
  if (write) GPTQ_LAUNCH((k_cache_write<T, KIND>), blocks, THREADS, 0, st, a, status);
  else GPTQ_LAUNCH((k_cache_read<T, KIND>), blocks, THREADS, 0, st, a, status);
  return GPTQ_OK;
}

template <typename T>
gptq_status by_kind(cudaStream_t st, bool write, int kind, Args& a, unsigned blocks, int32_t* status) {
  const auto off = [](const void* p, int64_t x, int64_t y) {
    return reinterpret_cast<uintptr_t>(p) | uintptr_t(x) * sizeof(T) | uintptr_t(y) * sizeof(T);
  };
  a.vec = 1;
  for (int i = 0; i < 2; ++i)
    if (off(write ? a.in[i] : a.out[i], a.ldt[i], a.heads > 1 ? a.ldh[i] : 0) & 15) a.vec = 0;
  if (kind == MX4) return launch<T, MX4>(st, write, a, blocks, status);
  if (kind == GRID8) return launch<T, GRID8>(st, write, a, blocks, status);
  return launch<T, GRID4>(st, write, a, blocks, status);
}

}  // namespace

bool cache_shape(const gptq_cache_config& cfg, int64_t dim, int& words, int& groups) {
  if (dim <= 0 || dim % 8 || dim > 4096) return false;
  if (cfg.kind == GPTQ_CACHE_MX) {
    if (cfg.group_size != 0 && cfg.group_size != 32) return false;
    groups = int((dim + 31) / 32);
    words = 4 * groups;
    return true;
  }
  const int g = cfg.group_size;
  if (g != 0 && g != 32 && g != 64 && g != 128) return false;
  if (g == 0 && dim > 256) return false;
  groups = g ? int((dim + g - 1) / g) : 1;
  words = int(dim * cfg.bits / 32);
  return true;
}

gptq_status cache_run(cudaStream_t st, bool write, const void* K, const void* V, int dtype,
                      int64_t tokens, int64_t k_ld_token, int64_t k_ld_head, int64_t v_ld_token,
                      int64_t v_ld_head, const gptq_cache_config& cfg, const gptq_cache& cache,
                      const gptq_cache_rows& rows, int32_t* status) {
  int words, groups, lane_bits = 0;
  if (!cache_shape(cfg, cache.dim, words, groups)) return GPTQ_ERR_UNSUPPORTED;
  const int units = int(cache.dim / 8);
  const int kind = cfg.kind == GPTQ_CACHE_MX ? MX4 : cfg.bits == 8 ? GRID8 : GRID4;
  const int per_group = kind == MX4 ? 4 : cfg.group_size ? cfg.group_size / 8 : units;
  while ((1 << lane_bits) < per_group) ++lane_bits;
  const int64_t per_head = int64_t(groups) << lane_bits, per_kv = per_head * cache.heads;
  if (2 * per_kv * MAX_ROWS > (int64_t(1) << 30)) return GPTQ_ERR_UNSUPPORTED;
  Args a{{K, V},
         {const_cast<void*>(K), const_cast<void*>(V)},
         {k_ld_token, v_ld_token},
         {k_ld_head, v_ld_head},
         {cache.k_codes, cache.v_codes},
         {cache.k_grids, cache.v_grids},
         {rows.table, rows.table_ld, rows.width, cache.pages, rows.cu, rows.start,
          int(rows.seqs), int(cache.page_size)},
         tokens, int(cache.heads), units, words, groups,
         lane_bits, 1, 0, cfg.sym, Div(uint32_t(2 * per_kv)), Div(uint32_t(per_kv)),
         Div(uint32_t(per_head))};
  // rows of a CTA: about STEPS units per thread, but no fewer CTAs than two per SM
  const int64_t fill = THREADS * STEPS / (2 * per_kv);
  a.rows = int(std::max<int64_t>(1, std::min<int64_t>({fill, tokens / (2 * 148), int64_t(MAX_ROWS)})));
  const int64_t blocks = (tokens + a.rows - 1) / a.rows;
  if (blocks > 0x7FFFFFFF) return GPTQ_ERR_UNSUPPORTED;
  switch (dtype) {
    case GPTQ_F32: return by_kind<float>(st, write, kind, a, unsigned(blocks), status);
    case GPTQ_F16: return by_kind<__half>(st, write, kind, a, unsigned(blocks), status);
    default: return by_kind<__nv_bfloat16>(st, write, kind, a, unsigned(blocks), status);
  }
}

}  // namespace gptq
