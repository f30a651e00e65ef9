// Index arithmetic of the paged key/value pools, for host and device: every
// address into a pool comes from here, after its bounds checks. Plain C++, so
// that it can be tested without a GPU.
#pragma once
#include <cstdint>

#if defined(__CUDACC__)
#define WSG_HD __host__ __device__ __forceinline__
#else
#define WSG_HD inline
#endif

namespace wsg {

constexpr int kPageSizeMax = 1024;

// A pool [num_pages][n_kv][1 << shift][head_dim] and the tables into it.
struct PagePool {
  int32_t num_pages, n_kv, shift;
  int32_t width;  // table entries per sequence (also the table's row stride)
};

// log2 of a page size, or -1 if it is not a power of two in [1, kPageSizeMax].
WSG_HD int page_shift(int page_size) {
  if (page_size < 1 || page_size > kPageSizeMax || (page_size & (page_size - 1))) return -1;
  int s = 0;
  while ((1 << s) < page_size) ++s;
  return s;
}

// Tokens a table row can hold.
WSG_HD int64_t page_capacity(const PagePool& p) { return static_cast<int64_t>(p.width) << p.shift; }

// The page that holds token `idx` of the sequence whose table row is `row`, or
// -1 (index outside the table, entry outside the pool).
WSG_HD int32_t page_of(const PagePool& p, const int32_t* row, int64_t idx) {
  if (idx < 0 || idx >= page_capacity(p)) return -1;
  const int32_t page = row[idx >> p.shift];
  return page >= 0 && page < p.num_pages ? page : -1;
}

// Row of head g, token idx inside the pool seen as [rows][head_dim], given its
// page (64 bits: pools pass 2^31 elements).
WSG_HD int64_t pool_row(const PagePool& p, int32_t page, int g, int64_t idx) {
  return ((static_cast<int64_t>(page) * p.n_kv + g) << p.shift) + (idx & ((int64_t{1} << p.shift) - 1));
}

}  // namespace wsg
