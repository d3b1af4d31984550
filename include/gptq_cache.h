/*
 * gptq_cache.h — a paged key/value cache in low-bit codes in libgptq.so: rows are quantised
 * as they are written and read back as floating point.
 *
 * The grids are those the library quantises weights with: a min-max integer grid per group
 * of values (gptq_quantize_layer; the GPTQ pages apply it to weights only), or the
 * microscaled 4-bit blocks of gptq_mx.h.  Here the values of one token and head, `dim` of
 * them, take the place of a weight row, and groups run along them:
 *   GPTQ_CACHE_GRID  bits 4 or 8; group_size 32, 64 or 128, or 0 for one group of all of
 *                    dim (dim <= 256); the last group may be shorter.  Per group, in IEEE
 *                    fp32: lo = min(0, values), hi = max(0, values); both 0: -1 and 1;
 *                        s = (hi - lo) / (2^bits - 1),  z = rint(-lo / s)
 *                    or with sym: m = max(-lo, hi) (1 if 0), s = 2m / (2^bits - 1),
 *                    z = 2^(bits-1).  code = clamp(rint(x / s) + z, 0, 2^bits - 1), which
 *                    stands for s (code - z).
 *   GPTQ_CACHE_MX    microscaled blocks of 32 (bits must be 4, group_size 0 or 32).
 * A group that holds a NaN or an infinity, or whose range overflows fp32, reads back as
 * NaN and raises GPTQ_ERR_NONFINITE in *dev_status; a group whose s underflows to 0 is
 * stored on the grid of [-1, 1].
 *
 * Stored form, slot = page * page_size + offset in it, G groups per head:
 *   codes  (slot * heads + head) * words + w, uint32 words in the bitstream of gptq_pack:
 *          words = ceil(dim * bits / 32) for GRID, 4 * ceil(dim / 32) for MX (codes past
 *          dim are 0)
 *   grids  GRID: fp32 pairs (s, z) at (slot * heads + head) * G + group; MX: one byte e.
 * Codes and grids 16-byte aligned; keys and values have arrays of their own.
 *
 * Rows and sequences.  A call's rows belong to sequences: rows cu[s] .. cu[s+1]-1 (cu holds
 * seqs + 1 non-decreasing entries; a sequence may have none) are positions start[s],
 * start[s] + 1, .. of sequence s, and position p lives in page table[s * table_ld + p /
 * page_size] at offset p % page_size.  Rows that belong to no sequence (at or past
 * cu[seqs]) are padding: a write ignores them and a read leaves them as they are.  A row whose position or page
 * is out of range (start < 0, p / page_size >= width, a page outside 0 .. pages-1) is left
 * out as well and raises GPTQ_ERR_INVALID_ARG in *dev_status; the other rows are done.
 * Two rows of one write must not have the same slot: what that slot holds is then not
 * defined (pages shared by sequences may be read, not written).
 *
 * Conventions are those of gptq.h.  A call launches at most one kernel, keeps no state,
 * needs no workspace and may be captured into a CUDA graph; cu, start and table are read
 * on the device when it runs.  A kernel may start while the call before it on the same
 * stream drains; it waits for that one's end before it touches memory.
 */
#ifndef GPTQ_CACHE_H_
#define GPTQ_CACHE_H_

#include "gptq.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { GPTQ_CACHE_GRID = 0, GPTQ_CACHE_MX = 1 };

typedef struct {
  int kind; /* GPTQ_CACHE_GRID or GPTQ_CACHE_MX */
  int bits;
  int group_size;
  int sym;
} gptq_cache_config;

/* The cache's arrays (device pointers) and their sizes. */
typedef struct {
  uint32_t* k_codes;
  void* k_grids;
  uint32_t* v_codes;
  void* v_grids;
  int64_t pages;
  int64_t page_size;
  int64_t heads;
  int64_t dim; /* a multiple of 8, at most 4096 */
} gptq_cache;

/* Which position of which sequence each row of a call is (device pointers). */
typedef struct {
  const int32_t* table;
  int64_t table_ld;
  int64_t width; /* pages per sequence in `table` */
  const int32_t* cu;
  const int32_t* start;
  int64_t seqs;
} gptq_cache_rows;

/* 32-bit words of codes, and bytes of grids, of one token and head (0: invalid or
 * unsupported cfg or dim). */
size_t gptq_cache_words(const gptq_cache_config* cfg, int64_t dim);
size_t gptq_cache_grid_bytes(const gptq_cache_config* cfg, int64_t dim);

/*
 * gptq_cache_write — quantise `tokens` rows of K and V into their slots.  K[t][h][0 .. dim-1]
 * is at K + t * k_ld_token + h * k_ld_head (elements, dtype), V alike; the rows may lie in
 * a larger buffer, in any order of strides.  Slots that no row has keep their contents.
 * tokens == 0 or seqs == 0 is a no-op.  Errors: INVALID_ARG, UNSUPPORTED (a group size or
 * dim that is not supported).
 */
gptq_status gptq_cache_write(const void* K, const void* V, int dtype, int64_t tokens,
                             int64_t k_ld_token, int64_t k_ld_head, int64_t v_ld_token,
                             int64_t v_ld_head, const gptq_cache_config* cfg,
                             const gptq_cache* cache, const gptq_cache_rows* rows,
                             int32_t* dev_status, void* stream);

/*
 * gptq_cache_read — the rows' values out of their slots into K and V (strides as above):
 * s (code - z), or level * 2^(e-127), formed in fp32 and rounded once to dtype.  The rows
 * of K and V must not overlap.  Errors as for gptq_cache_write.
 */
gptq_status gptq_cache_read(const gptq_cache_config* cfg, const gptq_cache* cache,
                            const gptq_cache_rows* rows, void* K, void* V, int dtype,
                            int64_t tokens, int64_t k_ld_token, int64_t k_ld_head,
                            int64_t v_ld_token, int64_t v_ld_head, int32_t* dev_status,
                            void* stream);

#ifdef __cplusplus
}
#endif
#endif /* GPTQ_CACHE_H_ */
