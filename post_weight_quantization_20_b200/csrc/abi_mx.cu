// The C ABI of the microscaled 4-bit rows (include/gptq_mx.h): argument checks and dispatch.
#include <atomic>
#include <climits>

#include "gptq_mx.h"
#include "kernels.h"

using namespace gptq;

static bool valid_dtype(int dt) { return dt == GPTQ_F32 || dt == GPTQ_F16 || dt == GPTQ_BF16; }
static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
static bool valid_shape(int64_t rows, int64_t cols) {
  return rows >= 0 && rows <= INT_MAX && cols > 0 && cols <= INT_MAX / 2;
}
// Rows and tokens of a product: indices of rows in a last tile of 256, and the number of tiles
// (256 rows x 64 tokens at the least), are ints.
static bool valid_product(int64_t rows, int64_t tokens) {
  return rows <= INT_MAX - 255 && tokens <= INT_MAX - 255 &&
         (rows + 255) / 256 * ((tokens + 63) / 64) <= int64_t(1) << 30;
}

static std::atomic<int32_t> g_give_up{-1};
namespace gptq {
int mx_give_up() { return g_give_up.load(std::memory_order_relaxed); }
}  // namespace gptq

extern "C" {

int32_t gptq_mx_debug_give_up(int32_t stages) {
  return g_give_up.exchange(stages < 0 ? -1 : stages, std::memory_order_relaxed);
}

size_t gptq_mx_scale_bytes(int64_t rows, int64_t cols) {
  if (!valid_shape(rows, cols)) return 0;
  return size_t((rows + 127) / 128) * size_t((cols + 127) / 128) * 512;
}

gptq_status gptq_mx_quantize(const void* X, int xdtype, int64_t rows, int64_t cols, int64_t ldx,
                             uint32_t* codes, uint8_t* scales, int32_t* dev_status, void* stream) {
  CallRange range_("gptq_mx_quantize");
  if (!valid_shape(rows, cols) || !valid_dtype(xdtype) || ldx < cols) return GPTQ_ERR_INVALID_ARG;
  if (rows == 0) return GPTQ_OK;
  if (!X || !codes || !scales || !aligned16(codes) || !aligned16(scales) ||
      !mx_grid_fits(rows, cols))
    return GPTQ_ERR_INVALID_ARG;
  return mx_quantize_run(as_stream(stream), X, xdtype, rows, int(cols), ldx, codes, scales,
                         dev_status);
}

gptq_status gptq_mx_dequantize(const uint32_t* codes, const uint8_t* scales, int64_t rows,
                               int64_t cols, void* Y, int ydtype, int64_t ldy, void* stream) {
  CallRange range_("gptq_mx_dequantize");
  if (!valid_shape(rows, cols) || !valid_dtype(ydtype) || ldy < cols) return GPTQ_ERR_INVALID_ARG;
  if (rows == 0) return GPTQ_OK;
  if (!Y || !codes || !scales || !aligned16(codes) || !aligned16(scales) ||
      !mx_grid_fits(rows, cols))
    return GPTQ_ERR_INVALID_ARG;
  return mx_dequantize_run(as_stream(stream), codes, scales, rows, int(cols), Y, ydtype, ldy);
}

gptq_status gptq_mx_matmul(const uint32_t* x_codes, const uint8_t* x_scales, int64_t m_tokens,
                           const uint32_t* w_codes, const uint8_t* w_scales, int64_t rows,
                           int64_t cols, void* Y, int ydtype, int64_t ldy, int32_t* dev_status,
                           void* stream) {
  CallRange range_("gptq_mx_matmul");
  if (!valid_shape(rows, cols) || !valid_shape(m_tokens, cols) || !valid_product(rows, m_tokens) ||
      !valid_dtype(ydtype) || ldy < rows)
    return GPTQ_ERR_INVALID_ARG;
  if (rows == 0 || m_tokens == 0) return GPTQ_OK;
  if (!x_codes || !x_scales || !w_codes || !w_scales || !Y || !aligned16(x_codes) ||
      !aligned16(x_scales) || !aligned16(w_codes) || !aligned16(w_scales))
    return GPTQ_ERR_INVALID_ARG;
  return mx_matmul_run(as_stream(stream), x_codes, x_scales, int(m_tokens), w_codes, w_scales,
                       int(rows), int(cols), Y, ydtype, ldy, dev_status);
}

}  // extern "C"
