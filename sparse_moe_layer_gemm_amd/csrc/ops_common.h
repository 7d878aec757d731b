// Device pieces of the operators around the layer: compile-time loops, NaN-keeping bf16 rounding,
// wavefront reductions and the map from a work item to an expert's rows.
#pragma once

#include <utility>

#include "device_common.h"
#include "ops_internal.h"

namespace moe {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

template <class F, int... I>
__device__ __forceinline__ void static_for_impl(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
// f(0) .. f(N - 1) with the index as a compile-time constant
template <int N, class F>
__device__ __forceinline__ void static_for(F&& f) {
  static_for_impl(f, std::make_integer_sequence<int, N>{});
}

// fp32 -> bf16, nearest even (hardware conversion: NaN stays NaN, overflow
// goes to infinity)
__device__ __forceinline__ uint32_t bf16_bits(float f) {
  return __builtin_bit_cast(uint16_t, (__bf16)f);
}
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const bf16x2 v = {(__bf16)lo, (__bf16)hi};
  return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ float bf16_lo(uint32_t d) { return __uint_as_float(d << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t d) { return __uint_as_float(d & 0xFFFF0000u); }

// Loads and stores of values that are used once: NT ones leave the caches to
// others. Elementwise calls take them when they move more than kStreamBytes (the
// caches hold 256 MB; what a small call writes, the next one finds there).
constexpr long long kStreamBytes = 128ll << 20;
template <bool NT, class T>
__device__ __forceinline__ T load_once(const T* p) {
  return NT ? __builtin_nontemporal_load(p) : *p;
}
template <bool NT, class T>
__device__ __forceinline__ void store_once(T* p, const T& v) {
  if constexpr (NT)
    __builtin_nontemporal_store(v, p);
  else
    *p = v;
}

// Rows [lo, lo + cnt) of expert e, with bounds outside [0, M] taken as 0 or M.
__device__ __forceinline__ void expert_rows(const int32_t* __restrict__ offsets, int e, int M,
                                            int& lo, int& cnt) {
  lo = min(max(offsets[e], 0), M);
  cnt = max(min(offsets[e + 1], M) - lo, 0);
}

// Source row of sorted row r, or -1 for a row of zeros.
__device__ __forceinline__ int source_row(const GroupedArgs& g, int r) {
  if (g.row_index == nullptr) return r;
  const int i = g.row_index[r];
  if (i < 0) return -1;
  const int s = g.row_div == 1 ? i : i / g.row_div;
  return s < g.a_rows ? s : -1;
}

// Sum over each lane's value in every lane (fixed butterfly order).
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
  return v;
}

}  // namespace
}  // namespace moe
