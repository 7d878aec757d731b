// Host checks shared by the entry points of the operators: limits, alignment,
// overlaps, and the sizes of a grouped product.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe.h"

namespace {

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxSorted = int64_t(1) << 29;  // rows of a grouped product (row indices stay below 2^31)
constexpr int32_t kMaxWidth = 1 << 20;            // K and N of a grouped product
constexpr int64_t kMaxBytes = int64_t(1) << 46;  // no array is larger than the address space
constexpr int64_t kMaxLanes = (int64_t(1) << 32) - 1;  // lanes of one grid dimension
constexpr int64_t kMaxTokens = int64_t(1) << 24;

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline moe_status launch_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH; }
inline bool is_float(int32_t d) { return d == MOE_F32 || d == MOE_BF16; }
inline int64_t elem(int32_t d) { return d == MOE_BF16 ? 2 : 4; }

// A required device array: present and 16-byte aligned.
inline bool array_ok(const void* p) { return p != nullptr && aligned16(p); }
// Whether [a, a + na) and [b, b + nb) intersect.
inline bool overlaps(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && na > 0 && nb > 0 && x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}
// rows * row_bytes, or -1 if it passes kMaxBytes
inline int64_t span(int64_t rows, int64_t row_bytes) {
  if (rows > 0 && row_bytes > kMaxBytes / rows) return -1;
  return rows * row_bytes;
}

inline moe_status check_grouped(int64_t a_rows, const int32_t* row_index, int32_t row_div, int64_t M,
                         int32_t K, int32_t N, int32_t E, int32_t k_unit) {
  if (M < 0 || K <= 0 || N <= 0 || E <= 0 || a_rows < 0) return MOE_ERR_INVALID_ARGUMENT;
  if (E > 256 || K % k_unit != 0 || N % 8 != 0 || K > kMaxWidth || N > kMaxWidth ||
      M >= kMaxSorted || a_rows > kMaxRows)
    return MOE_ERR_UNSUPPORTED;
  if (row_index) {
    if (row_div < 1) return MOE_ERR_INVALID_ARGUMENT;
  } else if (a_rows < M) {
    return MOE_ERR_INVALID_ARGUMENT;
  }
  return MOE_OK;
}

}  // namespace
