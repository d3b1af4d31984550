// Microscaled 4-bit rows: quantisation and read-back (include/gptq_mx.h).
//
// Both are one pass over the data, bound by HBM: 2 or 4 bytes per element on one side,
// 4.25 bits on the other.  A warp takes SPAN columns of one row, 8 columns (16 or 32 bytes)
// per lane and step, all of its loads first; a block's maximum is two shuffles among 4
// lanes, its codes one 32-bit word per lane, and the scales of 4 blocks one 32-bit store.
#include <algorithm>

#include "kernels.h"
#include "mx.cuh"

namespace gptq {
namespace {

constexpr int WARPS = 8;
constexpr int STEPS = 4;               // units of a lane per item, loaded together
constexpr int SPAN = STEPS * 32 * 8;   // columns of an item

template <typename T>
__global__ void __launch_bounds__(WARPS * 32)
k_mx_quantize(const T* __restrict__ X, int64_t rows, int cols, int64_t ldx, int spans, int vec,
              uint32_t* __restrict__ codes, uint8_t* __restrict__ scales, int32_t* status) {
  const int lane = threadIdx.x & 31;
  const int64_t item = int64_t(blockIdx.x) * WARPS + (threadIdx.x >> 5);
  const int64_t row = item / spans;
  if (row >= rows) return;
  const int c0 = int(item - row * spans) * SPAN;
  const int nb = (cols + 31) >> 5, ct = (nb + 3) >> 2;
  const T* x = X + row * ldx;
  Raw8<T> raw[STEPS];
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int c = c0 + (s * 32 + lane) * 8;
    load8(x + c, cols - c, vec != 0, raw[s]);
  }
  bool bad = false;
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int c = c0 + (s * 32 + lane) * 8, k = c >> 5;
    float v[8];
    widen8(raw[s], v);
    uint32_t m = mx::amax_bits8(v);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const int e = mx::scale_byte(m);
    uint32_t w = 0;
    if (e != 255) {
      const float f = mx::inv_scale(e);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= f;
      w = mx::encode8(v);
    } else {
      bad = true;
    }
    if (k < nb) codes[row * (4 * int64_t(nb)) + (c >> 3)] = w;
    // the bytes of 4 neighbouring blocks (16 lanes) as one word of their tile
    uint32_t q = uint32_t(e) << (8 * (k & 3));
    q |= __shfl_xor_sync(0xffffffffu, q, 4);
    q |= __shfl_xor_sync(0xffffffffu, q, 8);
    if ((lane & 15) == 0 && k < nb)
      *reinterpret_cast<uint32_t*>(scales + mx::scale_offset(row, k, ct)) = q;
  }
  if (bad) raise_status(status, GPTQ_ERR_NONFINITE);
}

template <typename T>
__global__ void __launch_bounds__(WARPS * 32)
k_mx_dequantize(const uint32_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                int64_t rows, int cols, int spans, int vec, T* __restrict__ Y, int64_t ldy) {
  const int lane = threadIdx.x & 31;
  const int64_t item = int64_t(blockIdx.x) * WARPS + (threadIdx.x >> 5);
  const int64_t row = item / spans;
  if (row >= rows) return;
  const int c0 = int(item - row * spans) * SPAN;
  const int nb = (cols + 31) >> 5, ct = (nb + 3) >> 2;
  uint32_t w[STEPS], e[STEPS];
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int c = c0 + (s * 32 + lane) * 8;
    w[s] = e[s] = 0;
    if (c < cols) {
      w[s] = __ldg(codes + row * (4 * int64_t(nb)) + (c >> 3));
      e[s] = __ldg(scales + mx::scale_offset(row, c >> 5, ct));
    }
  }
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int c = c0 + (s * 32 + lane) * 8;
    if (c >= cols) break;
    float v[8];
    mx::decode8(w[s], v);
    const float f = mx::scale_value(e[s]);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= f;
    store8(Y + row * ldy + c, cols - c, vec != 0, v);
  }
}

// vector accesses need every row to start on a 16-byte boundary
template <typename T>
int rows_aligned(const void* p, int64_t ld) {
  return ((reinterpret_cast<uintptr_t>(p) | uintptr_t(ld) * sizeof(T)) & 15) == 0;
}

template <typename T>
gptq_status quantize_t(cudaStream_t st, const void* X, int64_t rows, int cols, int64_t ldx,
                       uint32_t* codes, uint8_t* scales, int32_t* status) {
  const int spans = (cols + SPAN - 1) / SPAN;
  const int64_t blocks = (rows * spans + WARPS - 1) / WARPS;
  GPTQ_LAUNCH(k_mx_quantize<T>, unsigned(blocks), WARPS * 32, 0, st, static_cast<const T*>(X),
              rows, cols, ldx, spans, rows_aligned<T>(X, ldx), codes, scales, status);
  return GPTQ_OK;
}

template <typename T>
gptq_status dequantize_t(cudaStream_t st, const uint32_t* codes, const uint8_t* scales,
                         int64_t rows, int cols, void* Y, int64_t ldy) {
  const int spans = (cols + SPAN - 1) / SPAN;
  const int64_t blocks = (rows * spans + WARPS - 1) / WARPS;
  GPTQ_LAUNCH(k_mx_dequantize<T>, unsigned(blocks), WARPS * 32, 0, st, codes, scales, rows, cols,
              spans, rows_aligned<T>(Y, ldy), static_cast<T*>(Y), ldy);
  return GPTQ_OK;
}

}  // namespace

bool mx_grid_fits(int64_t rows, int64_t cols) {
  const int64_t spans = (cols + SPAN - 1) / SPAN;
  return rows * spans <= (int64_t(1) << 31) * WARPS - WARPS;
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
