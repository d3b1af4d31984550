/*
 * gptq_mx.h — microscaled 4-bit rows in libgptq.so: quantisation, read-back and the
 * product of two such matrices on the fifth-generation tensor cores.
 *
 * A row of a matrix (a weight's row, one token's activations) is cut into blocks of 32
 * consecutive columns.  A block shares one scale 2^(e-127), e = 0 .. 254 (255: the block
 * is not a number); an element is a 4-bit code: sign << 3 | magnitude, the magnitudes
 * 0 .. 7 standing for 0, 0.5, 1, 1.5, 2, 3, 4, 6 (one sign, two exponent, one mantissa
 * bit).  The GPTQ pages store integer grids only (gptq_quantize_layer); this is the
 * 4-bit form that the tensor cores multiply without a dequantisation step.
 *
 * Stored form of a rows x cols matrix, nb = ceil(cols / 32) blocks per row:
 *  codes   rows x 4*nb uint32 words, the bitstream of gptq_pack with 4-bit fields: column
 *          c in bits [4 (c % 8), 4 (c % 8) + 4) of word c / 8.  Codes at and past `cols`
 *          in a row's last block are 0.  16-byte aligned.
 *  scales  one byte e per block, in tiles of 128 rows x 4 blocks (512 bytes, the order
 *          in which the tensor cores take them): the byte of row r, block k is at
 *              ((r / 128) * ceil(nb / 4) + k / 4) * 512
 *                  + (r % 32) * 16 + ((r % 128) / 32) * 4 + k % 4,
 *          gptq_mx_scale_bytes() bytes in all.  For every row below `rows` the bytes of
 *          the blocks nb .. 4*ceil(nb/4)-1 are 0; bytes of rows past the last one are
 *          never written, and may hold anything.  16-byte aligned.
 *
 * Conventions (ownership, streams, status codes, device conditions) are those of gptq.h.
 * Every call launches at most one kernel, keeps no state and needs no workspace; results
 * do not depend on timing.  The calls may be captured into a CUDA graph.  A kernel may start
 * while the call before it on the same stream drains; it waits for that one's end before it
 * touches memory, so the order of the stream holds.
 */
#ifndef GPTQ_MX_H_
#define GPTQ_MX_H_

#include "gptq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of the scales of a rows x cols matrix (0 for rows < 0 or cols <= 0). */
size_t gptq_mx_scale_bytes(int64_t rows, int64_t cols);

/*
 * gptq_mx_quantize — the stored form of X (rows x cols, row stride ldx elements, xdtype).
 * Per block: e = max(0, E - 2) with E the biased fp32 exponent of the largest magnitude
 * (so that it lies in [4, 8) scales; a block of zeros gets e = 0); code = the level
 * nearest to x / 2^(e-127), ties to the even code, magnitudes above 6 to 6.  A block that
 * holds a NaN or an infinity gets e = 255 and codes 0, and raises GPTQ_ERR_NONFINITE in
 * *dev_status (may be NULL).  A row whose cols is not a multiple of 32 ends in a shorter
 * block.  rows == 0 is a no-op.  Errors: INVALID_ARG.
 */
gptq_status gptq_mx_quantize(const void* X, int xdtype, int64_t rows, int64_t cols, int64_t ldx,
                             uint32_t* codes, uint8_t* scales, int32_t* dev_status, void* stream);

/*
 * gptq_mx_dequantize — Y = the values the stored form stands for, level * 2^(e-127), formed
 * in fp32 and rounded once to ydtype (NaN where e = 255).  Y is rows x cols, row stride
 * ldy elements; elements of Y between cols and ldy are left as they are.
 * Errors: INVALID_ARG.
 */
gptq_status gptq_mx_dequantize(const uint32_t* codes, const uint8_t* scales, int64_t rows,
                               int64_t cols, void* Y, int ydtype, int64_t ldy, void* stream);

/*
 * gptq_mx_matmul — Y = X W^T of two stored forms: X m_tokens x cols (x_codes, x_scales), W
 * rows x cols (w_codes, w_scales), Y m_tokens x rows with row stride ldy elements, ydtype.
 *     Y[t][r] = sum_c x[t][c] w[r][c]
 * Products are exact, sums are held in fp32 and rounded once to ydtype.  Scales reach further
 * than fp32 does, from 2^-254 to 2^254 for a pair of blocks: what of a product or a sum lies
 * below 2^-149, fp32's least subnormal, is cut off; a sum beyond fp32's range is an infinity,
 * and NaN once infinities of both signs have met.  Any m_tokens, rows
 * from 0 (a no-op) to 2^31 - 256, not more than 2^30 tiles of 64 x 256 in all, and cols >= 1;
 * one token is as good a case as many.  A block of either
 * side with e = 255 makes the outputs of its row NaN.  Device conditions: TIMEOUT.
 * Errors: INVALID_ARG, UNSUPPORTED (the driver cannot encode the operands' tensor maps).
 */
gptq_status gptq_mx_matmul(const uint32_t* x_codes, const uint8_t* x_scales, int64_t m_tokens,
                           const uint32_t* w_codes, const uint8_t* w_scales, int64_t rows,
                           int64_t cols, void* Y, int ydtype, int64_t ldy, int32_t* dev_status,
                           void* stream);

/*
 * Diagnostic: in products launched after this call the MMA issuer of the last CTA (or CTA pair)
 * of every cluster gives up when it comes to its stage number `stages` of a tile, with the
 * copies and MMAs of the stages before it in flight; -1, the default, restores normal work.
 * The call then reports TIMEOUT and its Y is not defined, as where a wait runs out
 * (gptq_debug_set_wait_limit), but at a known place: so a test can check that CTAs which share
 * a tile's columns stop together, wait for what they have in flight and leave the context
 * usable.  Process-wide; returns the previous value.
 */
int32_t gptq_mx_debug_give_up(int32_t stages);

#ifdef __cplusplus
}
#endif
#endif /* GPTQ_MX_H_ */
