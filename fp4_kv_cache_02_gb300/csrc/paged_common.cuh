// paged_common.cuh -- the page table and the ragged batch, as the kernels of
// the paged cache see them.
//
// Entry e of sequence b is row e % page of page table[b][e / page] of the pool
// ("DeepSeek-V4.1-Flash: Pushing the Limits of KV Cache Compression" describes
// the entries, section 2.4.4; the pages are a server's way to hold many
// sequences of unknown lengths).
#pragma once

#include "common.cuh"

namespace csa2 {

struct PageTable {
  const int32_t* table;  // [B][max_pages]
  int64_t n_pages;       // pages of the pool
  int32_t max_pages;     // places of a sequence in the table
  int32_t shift;         // log2(page size)

  __host__ __device__ int32_t page_size() const { return 1 << shift; }
  // entries a sequence's places can hold (int32 counts: at most 2^31 - 1)
  __host__ __device__ int64_t capacity() const {
    const int64_t c = (int64_t)max_pages << shift;
    return c < 0x7FFFFFFFLL ? c : 0x7FFFFFFFLL;
  }
  // the pool's row of entry e of sequence b, -1 for a page outside the pool;
  // 0 <= e < capacity()
  __device__ __forceinline__ int64_t row(int32_t b, int64_t e) const {
    const int32_t page = table[(int64_t)b * max_pages + (e >> shift)];
    if (page < 0 || page >= n_pages) return -1;
    return ((int64_t)page << shift) + (e & (page_size() - 1));
  }
};

// A sequence's token rows [first, first + count); count -1 for a run that is
// not within 0 .. n_tokens.
struct TokenRun {
  int32_t first, count;
};
__device__ __forceinline__ TokenRun token_run(const int32_t* cu, int32_t b, int32_t n_tokens, int32_t per_seq) {
  if (!cu) return {b * per_seq, per_seq};
  const int32_t lo = cu[b], hi = cu[b + 1];
  if (lo < 0 || hi < lo || hi > n_tokens) return {0, -1};
  return {lo, hi - lo};
}

// Host side of the conventions of the paged entry points.
static inline int paged_check(const int32_t* page_table, int64_t n_pages, int32_t page_size, int32_t max_pages,
                              int32_t B, PageTable& pt) {
  if (n_pages < 0 || max_pages < 0 || page_size <= 0 || B < 0) return CSA2_ERR_INVALID_ARG;
  if (!page_table && B != 0 && max_pages != 0) return CSA2_ERR_INVALID_ARG;
  if (page_size < CSA2_MIN_PAGE || (page_size & (page_size - 1))) return CSA2_ERR_UNSUPPORTED_SHAPE;
  int32_t shift = 0;
  while ((1 << shift) < page_size) ++shift;
  if (n_pages > (0x7FFFFFFFLL >> shift)) return CSA2_ERR_UNSUPPORTED_SHAPE;
  if (!csa2_aligned(page_table, 4)) return CSA2_ERR_ALIGNMENT;
  pt = {page_table, n_pages, max_pages, shift};
  return CSA2_OK;
}

// The planes of a pool; one without pages has none (an empty tensor's address is null).
static inline bool paged_planes(int64_t n_pages, const void* data, const void* scale) {
  return n_pages == 0 || (data && scale);
}

// Rows of each sequence when cu is NULL.
static inline int paged_runs(const int32_t* cu, int32_t n_tokens, int32_t B, int32_t& per_seq) {
  per_seq = 0;
  if (n_tokens < 0 || B < 0) return CSA2_ERR_INVALID_ARG;
  if (!csa2_aligned(cu, 4)) return CSA2_ERR_ALIGNMENT;
  if (cu || B == 0) return CSA2_OK;
  if (n_tokens % B) return CSA2_ERR_INVALID_ARG;
  per_seq = n_tokens / B;
  return CSA2_OK;
}

}  // namespace csa2
