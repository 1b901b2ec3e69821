// api_util.h -- host helpers shared by the translation units that implement
// the C ABI.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <initializer_list>

#include "../../include/moeperm.h"
#include "common.cuh"

namespace moeperm {

constexpr int kMaxK = 32;
constexpr int kMaxL = 1024;
constexpr int64_t kMaxAssignments = int64_t(1) << 20;
constexpr int kMaxHidden = 32768;   // one pass of 2 chunks x 1024 threads per row
constexpr size_t kWsHeader = 256;  // reserved header before the chunk table

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// (NULL is aligned: whether it is allowed is another check)
inline bool aligned_to(const void* p, int n) { return reinterpret_cast<uintptr_t>(p) % (unsigned)n == 0; }

// Vectors of 32-bit elements that kernels read or write one element at a time.
inline bool words_ok(std::initializer_list<const void*> v) {
  for (const void* p : v)
    if (!aligned_to(p, 4)) return false;
  return true;
}

inline int num_sms_cached() {
  int n = 0;
  return device_attr_cached(cudaDevAttrMultiProcessorCount, &n) == cudaSuccess ? n : 0;
}

inline moe_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

// Bytes of an element type that rows move in (0: not one of them).
inline int elem_bytes(int type) {
  return type == MOE_BF16 || type == MOE_F16 ? 2 : type == MOE_F32 ? 4 : 0;
}
// A row of H elements starts and ends on 16 bytes, with the given row stride.
inline bool rows_ok(const void* p, int64_t ld, int32_t H, int es) {
  return p != nullptr && aligned16(p) && ld >= H && (ld * es) % 16 == 0;
}

}  // namespace moeperm
