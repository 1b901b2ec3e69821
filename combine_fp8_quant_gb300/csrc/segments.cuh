// segments.cuh -- where an expert's rows are, for the kernels that work on them:
// segments of a layout, slabs of `cap` rows, or one dense matrix.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace moeperm {

// First row and count of expert e (any kernel arguments with seg_begin, seg_end,
// cap and R). False for rows outside [0, R): nothing of them is read or written.
template <typename Args>
__device__ __forceinline__ bool segment(const Args& p, int e, int64_t& b, int64_t& c) {
  b = 0;
  c = p.R;
  if (p.cap > 0) {
    b = (int64_t)e * p.cap;
    c = __ldg(p.seg_end + e);
  } else if (p.seg_begin != nullptr) {
    b = __ldg(p.seg_begin + e);
    c = (int64_t)__ldg(p.seg_end + e) - b;
  }
  if (b >= 0 && c >= 0 && b + c <= p.R && !(p.cap > 0 && c > p.cap)) return true;
  b = c = 0;
  return false;
}

// What a count adds to the rows held, in kTermsByRows: any above the limit of all
// experts together decides alone, so a sum of 1024 stays within 32 bits.
__device__ __forceinline__ int rows_held(int64_t c) {
  constexpr int64_t kMost = (int64_t)kTwoTermRows * 1024 + 1;
  return (int)(c < kMost ? c : kMost);
}
__device__ __forceinline__ int terms_of(int held, int L) { return held <= kTwoTermRows * L ? 2 : 1; }

// Whether two segments have a row in common.
__device__ __forceinline__ bool share_rows(int64_t b0, int64_t c0, int64_t b1, int64_t c1) {
  return c0 > 0 && c1 > 0 && b0 < b1 + c1 && b1 < b0 + c0;
}

}  // namespace moeperm
