// Microscaled 4-bit rows: quantisation and read-back (include/gptq_mx.h).
//
// Both are one pass over the data, bound by HBM: 2 or 4 bytes per element on one side,
// 4.25 bits on the other.  A lane holds 32 bytes of a row to quantise (a block's maximum is
// one or two shuffles), or writes 16 bytes read back; a warp's steps are loaded together.
// Rows that are narrower than a warp's step share it, 2^lane_bits lanes to a row.
// Rows that do not start on 16-byte boundaries are still read and written in whole 16-byte
// granules, their bytes or codes shifted into place: element by element they took 6 to 7 times
// as long (20000 x 11003 bf16 read back: 609 us; through shared memory 236 us).
#include <algorithm>

#include "kernels.h"
#include "mx.cuh"

namespace gptq {
namespace {

constexpr int WARPS = 8;

struct Walk {
  int64_t rows;
  int cols;
  int lane_bits;      // narrow rows: a row takes 2^lane_bits lanes of a step
  int spans;          // wide rows: items of a row
  int64_t items;
};

// Which columns of which rows a warp's lanes take, step by step, N elements a lane.  Wide rows:
// consecutive steps of one row; narrow ones (WIDE false): 32 >> lane_bits rows a step.
template <int N, int STEPS, bool WIDE>
struct Item {
  int64_t row0;
  int col0, step;     // of step 0; rows (narrow) or columns (wide) per step
  __device__ Item(const Walk& w, int64_t item, int lane) {
    if (WIDE) {
      row0 = item / w.spans;
      col0 = int(item - row0 * w.spans) * (STEPS * 32 * N) + lane * N;
      step = 32 * N;
    } else {
      step = 32 >> w.lane_bits;
      row0 = item * (STEPS * step) + (lane >> w.lane_bits);
      col0 = (lane & ((1 << w.lane_bits) - 1)) * N;
    }
  }
  __device__ __forceinline__ int64_t row(int s) const { return WIDE ? row0 : row0 + s * step; }
  __device__ __forceinline__ int col(int s) const { return WIDE ? col0 + s * step : col0; }
};

template <typename T, bool VEC, bool WIDE>
__global__ void __launch_bounds__(WARPS * 32)
k_mx_quantize(const T* X, int64_t ldx, const Walk w, uint32_t* codes,
              uint8_t* scales, int32_t* status) {
  using U = Unit<T>;
  constexpr int STEPS = sizeof(T) == 4 ? 4 : 2;
  allow_successor();
  const int lane = threadIdx.x & 31;
  const int64_t item = int64_t(blockIdx.x) * WARPS + (threadIdx.x >> 5);
  wait_for_predecessor();
  if (item >= w.items) return;
  const Item<U::N, STEPS, WIDE> it(w, item, lane);
  const int nb = (w.cols + 31) >> 5, ct = (nb + 3) >> 2;
  const T* end = X + (w.rows - 1) * ldx + w.cols;
  U unit[STEPS];
  uint4 q2[VEC ? 1 : STEPS];
  bool whole[VEC ? 1 : STEPS];
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int64_t row = it.row(s);
    const int c = it.col(s), n = WIDE || row < w.rows ? w.cols - c : 0;
    const T* p = X + row * ldx + c;
    if constexpr (VEC) unit[s].load(p, n, true);
    else whole[s] = unit[s].begin(p, n, X, end, q2[s]);
  }
  bool bad = false;
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int64_t row = it.row(s);
    const int c = it.col(s), k = c >> 5;
    if constexpr (!VEC) unit[s].finish(X + row * ldx + c, whole[s], q2[s]);
    uint32_t m = unit[s].amax_bits();
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    if (U::N == 8) m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const int e = mx::scale_byte(m);
    float v[U::N];
    unit[s].widen(v);
    uint32_t q[U::WORDS];
    const float f = mx::inv_scale(min(e, 253));
#pragma unroll
    for (int i = 0; i < U::N; ++i) v[i] *= f;
#pragma unroll
    for (int j = 0; j < U::WORDS; ++j) q[j] = e == 255 ? 0u : mx::encode8(v + 8 * j);
    const bool live = (WIDE || row < w.rows) && k < nb;
    bad |= e == 255;
    if (live) {
      uint32_t* p = codes + row * (4 * int64_t(nb)) + (c >> 3);
      if constexpr (U::WORDS == 2) *reinterpret_cast<uint2*>(p) = make_uint2(q[0], q[1]);
      else *p = q[0];
    }
    // the bytes of 4 neighbouring blocks (8 or 16 lanes) as one word of their tile
    constexpr int BL = 32 / U::N;                        // lanes of a block
    uint32_t b = uint32_t(e) << (8 * (k & 3));
    b |= __shfl_xor_sync(0xffffffffu, b, BL);
    b |= __shfl_xor_sync(0xffffffffu, b, 2 * BL);
    if ((lane & (4 * BL - 1)) == 0 && live)
      *reinterpret_cast<uint32_t*>(scales + mx::scale_offset(row, k, ct)) = b;
  }
  if (bad) raise_status(status, GPTQ_ERR_NONFINITE);
}

// VEC: every row of Y starts on a 16-byte boundary.  Otherwise the lanes' units are moved back
// within each row to the boundaries there are: a unit then starts `shift` columns earlier, its
// codes straddle two words and perhaps two blocks, and its store is whole all the same.
template <typename T, bool VEC, bool WIDE>
__global__ void __launch_bounds__(WARPS * 32)
k_mx_dequantize(const uint32_t* codes, const uint8_t* scales, const Walk w,
                T* Y, int64_t ldy) {
  using O = Out<T>;
  constexpr int STEPS = 4;
  allow_successor();
  const int lane = threadIdx.x & 31;
  const int64_t item = int64_t(blockIdx.x) * WARPS + (threadIdx.x >> 5);
  wait_for_predecessor();
  if (item >= w.items) return;
  const Item<O::N, STEPS, WIDE> it(w, item, lane);
  const int nb = (w.cols + 31) >> 5, ct = (nb + 3) >> 2;
  uint32_t q[STEPS], q1[VEC ? 1 : STEPS], e[STEPS], e1[VEC ? 1 : STEPS];
  const auto shift = [&](int64_t row) {
    return VEC ? 0 : int(reinterpret_cast<uintptr_t>(Y + row * ldy) & 15) / int(sizeof(T));
  };
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int64_t row = it.row(s);
    const int c = it.col(s) - shift(row);
    q[s] = e[s] = 0;
    if constexpr (!VEC) q1[s] = e1[s] = 0;
    if (WIDE || row < w.rows) {
      const uint32_t* p = codes + row * (4 * int64_t(nb));
      if (VEC) {
        if (c < w.cols) {
          q[s] = p[c >> 3];
          e[s] = scales[mx::scale_offset(row, c >> 5, ct)];
        }
      } else {
        const int last = c + O::N - 1;
        if (c >= 0 && c < w.cols) {
          q[s] = p[c >> 3];
          e[s] = scales[mx::scale_offset(row, c >> 5, ct)];
        }
        if (last >= 0 && last < 32 * nb) {
          q1[s] = p[last >> 3];
          e1[s] = scales[mx::scale_offset(row, last >> 5, ct)];
        }
      }
    }
  }
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int64_t row = it.row(s);
    const int c = it.col(s) - shift(row);
    float v[O::N];
    uint32_t w0 = q[s];
    // the unit's codes as the lowest bits of one word
    if constexpr (!VEC) w0 = __funnelshift_r(q[s], q1[s], 4 * (c & 7));
    else if (O::N == 4) w0 >>= 4 * (c & 4);
    mx::decode<O::N>(w0, v);
    const float f = mx::scale_value(e[s]);
    const float f1 = VEC ? f : mx::scale_value(e1[VEC ? 0 : s]);
    const int own = 32 - (c & 31);                      // elements of the unit's first block
#pragma unroll
    for (int i = 0; i < O::N; ++i) v[i] *= VEC || i < own ? f : f1;
    T* p = Y + row * ldy + c;
    const int n = WIDE || row < w.rows ? w.cols - c : 0;
    if constexpr (VEC) O::store(p, n, true, v);
    else O::store_some(p, -c, n, v);
  }
}

// vector accesses need every row to start on a 16-byte boundary
template <typename T>
bool rows_aligned(const void* p, int64_t ld, int64_t rows) {
  return ((reinterpret_cast<uintptr_t>(p) | (rows > 1 ? uintptr_t(ld) * sizeof(T) : 0)) & 15) == 0;
}

// `reach`: columns of a row that the lanes have to cover; `least`: lane_bits of the narrowest
// row (4 blocks, whose scales are stored together)
Walk walk_of(int64_t rows, int cols, int reach, int n, int steps, int least) {
  Walk w{rows, cols, 5, 1, 0};
  const int lanes = ((reach + 31) / 32 * 32 + n - 1) / n;
  if (lanes <= 16) {
    w.lane_bits = least;
    while ((1 << w.lane_bits) < lanes) ++w.lane_bits;
  }
  if (w.lane_bits == 5) {
    w.spans = int((int64_t(reach) + steps * 32 * n - 1) / (steps * 32 * n));
    w.items = rows * w.spans;
  } else {
    const int64_t per = int64_t(steps) << (5 - w.lane_bits);
    w.items = (rows + per - 1) / per;
  }
  return w;
}

template <typename T, bool VEC>
gptq_status quantize_v(cudaStream_t st, const T* x, int64_t ldx, const Walk& w, uint32_t* codes,
                       uint8_t* scales, int32_t* status) {
  const unsigned blocks = unsigned((w.items + WARPS - 1) / WARPS);
  if (w.lane_bits == 5)
    GPTQ_LAUNCH_EARLY((k_mx_quantize<T, VEC, true>), blocks, WARPS * 32, st, x, ldx, w, codes, scales, status);
  else
    GPTQ_LAUNCH_EARLY((k_mx_quantize<T, VEC, false>), blocks, WARPS * 32, st, x, ldx, w, codes, scales, status);
  return GPTQ_OK;
}

template <typename T, bool VEC>
gptq_status dequantize_v(cudaStream_t st, const uint32_t* codes, const uint8_t* scales, const Walk& w,
                         T* y, int64_t ldy) {
  const unsigned blocks = unsigned((w.items + WARPS - 1) / WARPS);
  if (w.lane_bits == 5)
    GPTQ_LAUNCH_EARLY((k_mx_dequantize<T, VEC, true>), blocks, WARPS * 32, st, codes, scales, w, y, ldy);
  else
    GPTQ_LAUNCH_EARLY((k_mx_dequantize<T, VEC, false>), blocks, WARPS * 32, st, codes, scales, w, y, ldy);
  return GPTQ_OK;
}

template <typename T>
gptq_status quantize_t(cudaStream_t st, const void* X, int64_t rows, int cols, int64_t ldx,
                       uint32_t* codes, uint8_t* scales, int32_t* status) {
  const Walk w = walk_of(rows, cols, cols, Unit<T>::N, sizeof(T) == 4 ? 4 : 2, sizeof(T) == 4 ? 4 : 3);
  const T* x = static_cast<const T*>(X);
  return rows_aligned<T>(X, ldx, rows) ? quantize_v<T, true>(st, x, ldx, w, codes, scales, status)
                                       : quantize_v<T, false>(st, x, ldx, w, codes, scales, status);
}

template <typename T>
gptq_status dequantize_t(cudaStream_t st, const uint32_t* codes, const uint8_t* scales,
                         int64_t rows, int cols, void* Y, int64_t ldy) {
  T* y = static_cast<T*>(Y);
  if (rows_aligned<T>(Y, ldy, rows))
    return dequantize_v<T, true>(st, codes, scales, walk_of(rows, cols, cols, Out<T>::N, 4, 0), y, ldy);
  const int wide = cols + Out<T>::N - 1;               // moved back by up to N - 1 columns
  return dequantize_v<T, false>(st, codes, scales, walk_of(rows, cols, wide, Out<T>::N, 4, 0), y, ldy);
}

}  // namespace

// an item is never less than 512 elements of one row, or a row
bool mx_grid_fits(int64_t rows, int64_t cols) {
  return rows * ((cols + 518) / 512) <= (int64_t(1) << 31) * WARPS - WARPS;
}

gptq_status mx_quantize_run(cudaStream_t st, const void* X, int dt, int64_t rows, int cols,
                            int64_t ldx, uint32_t* codes, uint8_t* scales, int32_t* status) {
  if (rows == 0) return GPTQ_OK;
  switch (dt) {
    case GPTQ_F32: return quantize_t<float>(st, X, rows, cols, ldx, codes, scales, status);
    case GPTQ_F16: return quantize_t<__half>(st, X, rows, cols, ldx, codes, scales, status);
    default: return quantize_t<__nv_bfloat16>(st, X, rows, cols, ldx, codes, scales, status);
  }
}

gptq_status mx_dequantize_run(cudaStream_t st, const uint32_t* codes, const uint8_t* scales,
                              int64_t rows, int cols, void* Y, int dt, int64_t ldy) {
  if (rows == 0) return GPTQ_OK;
  switch (dt) {
    case GPTQ_F32: return dequantize_t<float>(st, codes, scales, rows, cols, Y, ldy);
    case GPTQ_F16: return dequantize_t<__half>(st, codes, scales, rows, cols, Y, ldy);
    default: return dequantize_t<__nv_bfloat16>(st, codes, scales, rows, cols, Y, ldy);
  }
}

}  // namespace gptq
