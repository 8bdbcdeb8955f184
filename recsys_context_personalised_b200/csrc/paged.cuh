// Index arithmetic of the paged key/value cache, shared by the kernels and by
// a host program that checks it on the CPU (no CUDA types in here).
//
// The cache holds pages of `page` rows per kv head: [num_pages, hk, page, dh].
// Row `pos` of sample b lies in page table[b * max_pages + pos / page] at row
// pos % page.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define GDPA_HD __host__ __device__ __forceinline__
#else
#define GDPA_HD inline
#endif

namespace gdpa {

// Page id of position `pos` (>= 0) of a sample whose table row is `row`, or -1
// when the position lies past the table or the entry names no page.
GDPA_HD int32_t page_of(const int32_t* row, int max_pages, int num_pages, int page_shift,
                        int64_t pos) {
  const int64_t slot = pos >> page_shift;
  if (pos < 0 || slot >= max_pages) return -1;
  const int32_t id = row[slot];
  return id >= 0 && id < num_pages ? id : -1;
}

// Element offset of (page, kv head, row) in a cache tensor.
GDPA_HD int64_t cache_row(int32_t id, int head, int hk, int page_shift, int row, int dh) {
  return ((((int64_t)id * hk + head) << page_shift) + row) * dh;
}

}  // namespace gdpa
