// Where a row of a cache call lives (include/gptq_cache.h, "Rows and sequences").  Plain
// C++, so that the index arithmetic also compiles and is tested on the host.
#pragma once
#include <stdint.h>

#ifdef __CUDACC__
#define GPTQ_HD __host__ __device__ __forceinline__
#else
#define GPTQ_HD inline
#endif

namespace gptq {

enum { SLOT_NONE = -1, SLOT_BAD = -2 };   // a padding row; a position or page out of range

struct RowMap {
  const int32_t* table;
  int64_t table_ld, width, pages;
  const int32_t* cu;
  const int32_t* start;
  int seqs, page_size;
};

// page * page_size + offset of row t (t >= 0, seqs >= 1), or SLOT_NONE or SLOT_BAD.  Reads cu
// inside 0 .. seqs, start inside 0 .. seqs-1 and table inside its rows and width, whatever
// they hold.
GPTQ_HD int64_t slot_of(const RowMap& m, int64_t t) {
  int lo = 0, hi = m.seqs;             // the last sequence whose first row is at or before t
  while (hi - lo > 1) {
    const int mid = lo + ((hi - lo) >> 1);
    if (m.cu[mid] <= t) lo = mid; else hi = mid;
  }
  const int64_t first = m.cu[lo];
  if (t < first || t >= m.cu[lo + 1]) return SLOT_NONE;
  const int64_t begin = m.start[lo], pos = begin + (t - first);
  const int64_t page_no = pos / m.page_size;
  if (begin < 0 || page_no >= m.width) return SLOT_BAD;
  const int64_t page = m.table[int64_t(lo) * m.table_ld + page_no];
  if (page < 0 || page >= m.pages) return SLOT_BAD;
  return page * m.page_size + (pos - page_no * m.page_size);
}

}  // namespace gptq
