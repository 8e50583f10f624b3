// device_input.cuh -- lengths and block-table entries that are read on the
// device: how one out of range is reported, and the checked page lookup.
#pragma once
#include <cstdint>

namespace lca {

constexpr int kErrInput = 4;          // device error word bit: a length or page entry out of range

__device__ __forceinline__ void input_error(int* err, int where) {
  if (atomicOr(err, kErrInput) == 0) atomicExch(err + 1, where);
}

// The pool row of token `tok` of sequence b: its page from the block table,
// checked against the pool (an entry outside [0, num_pages) raises the device
// input bit, and page 0 is read instead, so no access leaves the pool).
__device__ __forceinline__ int64_t paged_row(const int32_t* table, int64_t row_stride, int page_size,
                                             int64_t num_pages, int64_t b, int64_t tok, int* err,
                                             int where) {
  const uint32_t ps = (uint32_t)page_size;
  const uint32_t t = (uint32_t)tok;
  const uint32_t j = t / ps;
  int64_t page = table[b * row_stride + j];
  if (page < 0 || page >= num_pages) {
    input_error(err, where);
    page = 0;
  }
  return page * page_size + (t - j * ps);
}

}  // namespace lca
