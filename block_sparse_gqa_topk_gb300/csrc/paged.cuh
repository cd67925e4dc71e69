// paged.cuh -- addressing of a paged cache, shared by the kernels that write and read it.
//
// The pool holds num_pages pages of page_size token rows; sequence b's token at position
// pos is row pos % page_size of page table[b][pos / page_size].  Page ids are read on the
// device, so each is checked there before it becomes an address.
#pragma once

#include "common.cuh"

namespace msa {

struct PageView {
  const int32_t* table;  // [B] rows of max_pages page ids
  int64_t table_stride;
  int num_pages, page_size, max_pages;
  int shift;  // log2(page_size), or -1
};

__device__ __forceinline__ int page_of(const PageView& v, int pos) {
  return v.shift >= 0 ? pos >> v.shift : pos / v.page_size;
}

// Pool row of a position 0 <= pos < max_pages * page_size; -1 where the table names no
// page of the pool.
__device__ __forceinline__ int64_t pool_row(const PageView& v, int b, int pos) {
  const int slot = page_of(v, pos);
  const int id = __ldg(&v.table[(int64_t)b * v.table_stride + slot]);
  if ((unsigned)id >= (unsigned)v.num_pages) return -1;
  return (int64_t)id * v.page_size + (pos - slot * v.page_size);
}

inline int page_shift(int page_size) {
  for (int s = 0; s < 31; ++s)
    if ((1 << s) == page_size) return s;
  return -1;
}

}  // namespace msa
