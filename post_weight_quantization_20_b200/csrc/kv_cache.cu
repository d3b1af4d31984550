// The paged low-bit key/value cache (include/gptq_cache.h): rows are quantised as they are
// written and read back as floating point.
//
// Both directions are one pass over the rows, bound by HBM (2 or 4 bytes per value on one
// side, 4.25 to 10 bits on the other) or, for a token per sequence, by the launch and the
// chain cu -> start -> table -> slot.  A lane takes 32 or 64 bytes of a row to quantise, and a
// group is 1 to 16 neighbouring lanes, so that its range is a few shuffles and nothing is staged; to
// read, a lane writes 16 bytes.  A thread's place in a row (K or V, head, group) is the same in
// every row that it takes, so it is worked out once.  One thread per row finds its sequence and
// slot, in a write while the first loads are in flight.
#include <algorithm>

#include "grid.cuh"
#include "kernels.h"
#include "kv_slots.h"
#include "mx.cuh"
#include "tc_common.cuh"

namespace gptq {
namespace {

constexpr int THREADS = 256;
constexpr int STEPS = 4;          // rows of a thread whose loads are issued together in a read

struct Args {
  const void* in[2];     // write: K and V
  void* out[2];          // read: K and V
  int64_t ldt[2], ldh[2];
  uint32_t* codes[2];
  void* grids[2];
  RowMap map;
  int64_t tokens;
  int heads, dim, words, groups;     // words and groups of one head
  int group;                         // values of a group
  int lane_bits;                     // write: a group is 2^lane_bits lanes
  int per_head, per_row;             // lanes of a head, and of a row (K and V)
  int side;                          // rows that a CTA takes side by side
  int rows;                          // rows of a CTA, at most THREADS
  int vec;                           // all rows on 16-byte boundaries
  int sym;
};

// What a thread works on in each of its rows: K or V, head, lane of the head.
struct Place {
  int row, kv, head, lane;
  bool live;
  __device__ explicit Place(const Args& a) {
    const int t = blockIdx.y * THREADS + threadIdx.x;      // per_row > THREADS: a part of one row
    row = t / a.per_row;
    int i = t - row * a.per_row;
    live = row < a.side;
    const int per_kv = a.per_row >> 1;
    kv = i >= per_kv;
    i -= kv ? per_kv : 0;
    head = i / a.per_head;
    lane = i - head * a.per_head;
  }
};

// Where row t is stored: its first word of codes and its first group, or negative if nowhere
// (reported by the first part of a row only).
struct Where {
  int64_t word, group;
};
__device__ __forceinline__ Where find_row(const Args& a, int64_t t, int32_t* status) {
  const int64_t slot = slot_of(a.map, t);
  if (slot == SLOT_BAD && blockIdx.y == 0) raise_status(status, GPTQ_ERR_INVALID_ARG);
  return {slot < 0 ? -1 : slot * (int64_t(a.heads) * a.words), slot * (int64_t(a.heads) * a.groups)};
}

enum { GRID4 = 0, GRID8 = 1, MX4 = 2 };

// x / s rounded to fp32 where nothing under- or overflows, without a division: inv + low is
// 1 / s to about 48 bits, so that the first q is within half an ulp and a little of the quotient,
// and from there one residual correction with inv, 1 / s rounded, gives the correctly rounded
// quotient (Markstein, IBM J. Res. Dev. 34(1), 1990: q within one ulp is enough).  The codes need
// that rounding: 16-bit values hit exact ties of their grid all the time (15 x / (hi - lo) is a
// fraction of small whole numbers).  With a division per value a write took 470 us (131072
// tokens of 8 x 128 bf16 K and V).
__device__ __forceinline__ float quotient(float x, float s, float inv, float low) {
  const float q = fmaf(x, inv, x * low);
  return fmaf(fmaf(-q, s, x), inv, q);
}
__device__ __forceinline__ float low_part(float s, float inv) { return fmaf(-inv, s, 1.f) * inv; }

enum { GRID_FAST = 0, GRID_SLOW = 1, GRID_NAN = 2 };

// The grid of [lo, hi] as grid_params defines it, and the codes clamp(rint(x / s) + z, 0, maxq) of
// values on it.
template <int maxq>
struct Grid {
  float s, z, inv, low;
  int zi, kind;
  __device__ __forceinline__ Grid(float lo, float hi, int sym) {
    const float m = fmaxf(-lo, hi);
    const float width = sym ? m + m : hi - lo;
    kind = GRID_FAST;
    inv = low = 0.f;
    zi = 0;
    if (width > 0x1p-90f && width < 0x1p90f) {   // no under- or overflow below (NaN is neither)
      constexpr float r = 1.f / float(maxq);     // rounded, and what that leaves of 1 / maxq
      constexpr float rl = float(1.0 / maxq - double(r));
      s = quotient(width, float(maxq), r, rl);
      inv = __frcp_rn(s);
      low = low_part(s, inv);
      zi = sym ? (maxq + 1) / 2 : whole(quotient(-lo, s, inv, low));
      z = sym ? float(zi) : copysignf(float(zi), -lo);   // a zero with the sign of rint(-lo / s)
      return;
    }
    kind = GRID_SLOW;
    grid_params(lo, hi, float(maxq), sym, s, z);
    if (s == 0.f) grid_params(-1.f, 1.f, float(maxq), sym, s, z);     // an underflowed range
    if (lo != lo || !(s <= 3.402823466e38f)) {
      kind = GRID_NAN;
      s = __uint_as_float(0x7FC00000u);
      z = 0.f;
    }
  }
  // rint(q) of |q| < 2^22: adding 1.5 * 2^23 rounds to a whole number, which is the sum's low bits
  static constexpr int MAGIC_BITS = 0x4B400000;
  static __device__ __forceinline__ int whole(float q) { return __float_as_int(q + 12582912.f) - MAGIC_BITS; }

  template <int N>
  __device__ __forceinline__ void codes(const float (&x)[N], int (&c)[N]) const {
    if (kind == GRID_FAST) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        c[i] = __vimin_s32_relu(__float_as_int(quotient(x[i], s, inv, low) + 12582912.f) + (zi - MAGIC_BITS), maxq);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        c[i] = kind == GRID_NAN ? 0 : int(fminf(fmaxf(rintf(__fdiv_rn(x[i], s)) + z, 0.f), float(maxq)));
    }
  }
};

// CTAs that an SM holds at once, and the most rounds of rows of one.  Measured on 131072 tokens of
// 8 x 128 bf16, grids, and 16384 of 32 x 128 fp16, blocks: reads 4 / 6 / 8 at once 130 / 124 / 143 us
// for grids, whose spills start at 8 as those of fp32 blocks do, and 101 / 81 / 69 us for blocks.
template <typename T, int KIND>
struct Resident {
  static constexpr int WRITE = KIND == MX4 ? 5 : 3, READ = KIND == MX4 && sizeof(T) == 2 ? 8 : 6;
};
constexpr int ROUNDS = 32;

// Units of a lane in a write.  A group's range, grid and addresses cost a lane about as many
// instructions as 16 codes do, and the kernel is bound by issuing them.
template <int KIND>
constexpr int LANE_UNITS = KIND == MX4 ? 1 : 2;

template <typename T, int KIND>
__global__ void __launch_bounds__(THREADS, Resident<T, KIND>::WRITE)
k_cache_write(const Args a, int32_t* status) {
  using U = Unit<T>;
  constexpr int LU = LANE_UNITS<KIND>, LN = LU * U::N;
  __shared__ Where stored[THREADS];
  allow_successor();
  const Place pl(a);
  wait_for_predecessor();
  const int64_t t0 = int64_t(blockIdx.x) * a.rows;
  const int rows = int(min(int64_t(a.rows), a.tokens - t0));
  const int group = pl.lane >> a.lane_bits;
  const int first = pl.lane * LN;                         // first value of the lane
  const int n = pl.live ? a.dim - first : 0;
  const T* in = static_cast<const T*>(a.in[pl.kv]) + (t0 + pl.row) * a.ldt[pl.kv] +
                pl.head * a.ldh[pl.kv] + first;
  const int64_t step = a.ldt[pl.kv] * a.side;
  uint32_t* codes0 = a.codes[pl.kv] + int64_t(pl.head) * a.words + first / (KIND == GRID8 ? 4 : 8);
  const int64_t group0 = int64_t(pl.head) * a.groups + group;
  bool bad = false;
  // the next row is loading while one is quantised (one copy of that code: unrolled over the
  // rows it no longer fits the instruction cache; loading two ahead cost 6% for its registers)
  U next[LU];
#pragma unroll
  for (int u = 0; u < LU; ++u)
    next[u].load(in + u * U::N, pl.row < rows ? n - u * U::N : 0, a.vec != 0);
  if (int(threadIdx.x) < rows) stored[threadIdx.x] = find_row(a, t0 + threadIdx.x, status);
  __syncthreads();
#pragma unroll 1
  for (int r0 = 0; r0 < rows; r0 += a.side) {
    U now[LU];
    const int r = r0 + pl.row;
    in += step;
#pragma unroll
    for (int u = 0; u < LU; ++u) {
      now[u] = next[u];
      next[u].load(in + u * U::N, r + a.side < rows ? n - u * U::N : 0, a.vec != 0);
    }
    Where at = {-1, 0};
    if (r < rows && pl.live) at = stored[r];
    uint32_t* codes = codes0 + at.word;
    if constexpr (KIND == MX4) {
      float v[U::N];
      now[0].widen(v);
      uint32_t m = now[0].amax_bits();
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      if (U::N == 8) m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const int e = mx::scale_byte(m);
      const float f = mx::inv_scale(min(e, 253));
      uint32_t w[U::WORDS];
#pragma unroll
      for (int j = 0; j < U::N; ++j) v[j] *= f;
#pragma unroll
      for (int j = 0; j < U::WORDS; ++j) w[j] = e == 255 ? 0u : mx::encode8(v + 8 * j);
      if (at.word >= 0) {
        bad |= e == 255;
        if constexpr (U::WORDS == 2) *reinterpret_cast<uint2*>(codes) = make_uint2(w[0], w[1]);
        else *codes = w[0];
        if ((first & 31) == 0)
          static_cast<uint8_t*>(a.grids[pl.kv])[at.group + group0] = uint8_t(e);
      }
    } else {
      constexpr int maxq = KIND == GRID4 ? 15 : 255;
      float lo, hi;
      now[0].range(lo, hi);
#pragma unroll
      for (int u = 1; u < LU; ++u) {
        float l, h;
        now[u].range(l, h);
        lo = min_nan(lo, l);
        hi = max_nan(hi, h);
      }
      for (int o = 1; o < (1 << a.lane_bits); o <<= 1) {
        lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
      }
      lo = min_nan(lo, 0.f);
      hi = max_nan(hi, 0.f);
      const Grid<maxq> g(lo, hi, a.sym);
      if (at.word >= 0 && n > 0) {
        bad |= g.kind == GRID_NAN;
        // 8 codes at a time: all of dim, which is a multiple of 8, and no more
#pragma unroll
        for (int u = 0; u < LU; ++u) {
          float v[U::N];
          int c[U::N];
          now[u].widen(v);
          g.template codes<U::N>(v, c);
#pragma unroll
          for (int j = 0; j < U::WORDS; ++j) {
            const int k = u * U::WORDS + j;              // eighth of the lane's values
            if constexpr (KIND == GRID4) {
              uint32_t w = 0;
#pragma unroll
              for (int i = 0; i < 8; ++i) w += uint32_t(c[8 * j + i]) << (4 * i);
              if (8 * k < n) codes[k] = w;
            } else {
              uint32_t w[2] = {0u, 0u};
#pragma unroll
              for (int i = 0; i < 8; ++i) w[i >> 2] += uint32_t(c[8 * j + i]) << (8 * (i & 3));
              if (8 * k < n) *reinterpret_cast<uint2*>(codes + 2 * k) = make_uint2(w[0], w[1]);
            }
          }
        }
        if (pl.lane == group << a.lane_bits)
          static_cast<float2*>(a.grids[pl.kv])[at.group + group0] = make_float2(g.s, g.z);
      }
    }
  }
  if (bad) raise_status(status, GPTQ_ERR_NONFINITE);
}

template <typename T, int KIND>
__global__ void __launch_bounds__(THREADS, Resident<T, KIND>::READ)
k_cache_read(const Args a, int32_t* status) {
  using O = Out<T>;
  __shared__ Where stored[THREADS];
  allow_successor();
  const Place pl(a);
  wait_for_predecessor();
  const int64_t t0 = int64_t(blockIdx.x) * a.rows;
  const int rows = int(min(int64_t(a.rows), a.tokens - t0));
  if (int(threadIdx.x) < rows) stored[threadIdx.x] = find_row(a, t0 + threadIdx.x, status);
  const int first = pl.lane * O::N;
  const int group = first / a.group;
  const uint32_t* codes = a.codes[pl.kv] + int64_t(pl.head) * a.words + first / (KIND == GRID8 ? 4 : 8);
  const int64_t group0 = int64_t(pl.head) * a.groups + group;
  T* out = static_cast<T*>(a.out[pl.kv]) + t0 * a.ldt[pl.kv] + pl.head * a.ldh[pl.kv] + first;
  const int64_t ldt = a.ldt[pl.kv];
  __syncthreads();
  if (!pl.live) return;
  for (int r0 = pl.row; r0 < rows; r0 += STEPS * a.side) {
    uint32_t w[STEPS][2], e[STEPS];
    float2 g[STEPS];
    bool live[STEPS];
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int r = r0 + s * a.side;
      Where at = {-1, 0};
      if (r < rows) at = stored[r];
      live[s] = at.word >= 0;
      if (!live[s]) continue;
      const uint32_t* p = codes + at.word;
      if constexpr (KIND == GRID8 && O::N == 8) {
        const uint2 q = *reinterpret_cast<const uint2*>(p);
        w[s][0] = q.x;
        w[s][1] = q.y;
      } else {
        w[s][0] = *p;
      }
      if constexpr (KIND == MX4)
        e[s] = static_cast<const uint8_t*>(a.grids[pl.kv])[at.group + group0];
      else
        g[s] = static_cast<const float2*>(a.grids[pl.kv])[at.group + group0];
    }
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      if (!live[s]) continue;
      float v[O::N];
      // 4 fp32 values of a head are half a word of 4-bit codes
      if (KIND != GRID8 && O::N == 4) w[s][0] >>= 4 * (first & 4);
      if constexpr (KIND == MX4) {
        // a scale that fp16 holds multiplies the levels there: both are exact, the product is
        // rounded once
        if constexpr (__is_same(T, __half)) {
          if (a.vec && e[s] - 103u <= 39u) {
            *reinterpret_cast<uint4*>(out + (r0 + s * a.side) * ldt) = mx::decode8_half(w[s][0], e[s]);
            continue;
          }
        }
        mx::decode<O::N>(w[s][0], v);
        const float f = mx::scale_value(e[s]);
#pragma unroll
        for (int j = 0; j < O::N; ++j) v[j] *= f;
      } else {
        // the code as a float without a conversion: 2^23 + c (the code as the lowest byte of
        // that float), less 2^23 + z; both are whole numbers below 2^24 (z < 2^10 on any grid
        // that a write stores), the difference exact
        const float zz = 8388608.f + g[s].y;
        if constexpr (KIND == GRID4) {             // even codes to bytes, odd ones to bytes
          w[s][1] = (w[s][0] >> 4) & 0x0F0F0F0Fu;
          w[s][0] &= 0x0F0F0F0Fu;
        }
#pragma unroll
        for (int j = 0; j < O::N; ++j) {
          const uint32_t from = KIND == GRID4 ? w[s][j & 1] : w[s][j >> 2];
          const uint32_t byte = KIND == GRID4 ? j >> 1 : j & 3;
          v[j] = g[s].x * (__uint_as_float(__byte_perm(from, 0x4B000000u, 0x7540u + byte)) - zz);
        }
      }
      O::store(out + (r0 + s * a.side) * ldt, O::N, a.vec != 0, v);
    }
  }
}

template <typename T, int KIND>
gptq_status launch(cudaStream_t st, bool write, Args& a, int32_t* status) {
  if (write) {
    constexpr int LN = LANE_UNITS<KIND> * Unit<T>::N;
    const int per_group = (a.group + LN - 1) / LN;
    while ((1 << a.lane_bits) < per_group) ++a.lane_bits;
    a.per_head = a.groups << a.lane_bits;
  } else {
    a.per_head = a.dim / Out<T>::N;
  }
  const int64_t per_row = int64_t(2) * a.heads * a.per_head;
  const int64_t parts = (per_row + THREADS - 1) / THREADS;
  if (parts > 65535) return GPTQ_ERR_UNSUPPORTED;
  a.per_row = int(per_row);
  a.side = std::max(1, THREADS / a.per_row);
  // rows of a CTA: as many as pay for finding their slots, in whole waves of resident CTAs
  // (a last wave that was three quarters full cost 15%)
  const int sms = sm_count();
  if (sms <= 0) return GPTQ_ERR_CUDA;
  const int64_t slots = int64_t(sms) * (write ? Resident<T, KIND>::WRITE : Resident<T, KIND>::READ);
  const int64_t work = a.tokens * parts, most = std::min(THREADS / a.side, ROUNDS) * a.side;
  const int64_t waves = (work + slots * most - 1) / (slots * most);
  const int64_t even = (work + slots * waves - 1) / (slots * waves);
  a.rows = int((even + a.side - 1) / a.side * a.side);
  const int64_t blocks = (a.tokens + a.rows - 1) / a.rows;
  const dim3 grid{unsigned(blocks), unsigned(parts)};
  if (write) GPTQ_LAUNCH_EARLY((k_cache_write<T, KIND>), grid, THREADS, st, a, status);
  else GPTQ_LAUNCH_EARLY((k_cache_read<T, KIND>), grid, THREADS, st, a, status);
  return GPTQ_OK;
}

template <typename T>
gptq_status by_kind(cudaStream_t st, bool write, int kind, Args& a, int32_t* status) {
  const auto off = [](const void* p, int64_t x, int64_t y) {
    return reinterpret_cast<uintptr_t>(p) | uintptr_t(x) * sizeof(T) | uintptr_t(y) * sizeof(T);
  };
  a.vec = 1;
  for (int i = 0; i < 2; ++i)
    if (off(write ? a.in[i] : a.out[i], a.tokens > 1 ? a.ldt[i] : 0, a.heads > 1 ? a.ldh[i] : 0) & 15)
      a.vec = 0;
  if (kind == MX4) return launch<T, MX4>(st, write, a, status);
  if (kind == GRID8) return launch<T, GRID8>(st, write, a, status);
  return launch<T, GRID4>(st, write, a, status);
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
  Args a = {};
  if (!cache_shape(cfg, cache.dim, a.words, a.groups)) return GPTQ_ERR_UNSUPPORTED;
  const int kind = cfg.kind == GPTQ_CACHE_MX ? MX4 : cfg.bits == 8 ? GRID8 : GRID4;
  a.in[0] = K;
  a.in[1] = V;
  a.out[0] = const_cast<void*>(K);
  a.out[1] = const_cast<void*>(V);
  a.ldt[0] = k_ld_token;
  a.ldt[1] = v_ld_token;
  a.ldh[0] = k_ld_head;
  a.ldh[1] = v_ld_head;
  a.codes[0] = cache.k_codes;
  a.codes[1] = cache.v_codes;
  a.grids[0] = cache.k_grids;
  a.grids[1] = cache.v_grids;
  a.map = {rows.table, rows.table_ld, rows.width, cache.pages, rows.cu, rows.start,
           int(rows.seqs), int(cache.page_size)};
  a.tokens = tokens;
  a.heads = int(cache.heads);
  a.dim = int(cache.dim);
  a.group = kind == MX4 ? 32 : cfg.group_size ? cfg.group_size : a.dim;
  a.sym = cfg.sym;
  switch (dtype) {
    case GPTQ_F32: return by_kind<float>(st, write, kind, a, status);
    case GPTQ_F16: return by_kind<__half>(st, write, kind, a, status);
    default: return by_kind<__nv_bfloat16>(st, write, kind, a, status);
  }
}

}  // namespace gptq
