// Device pieces of routing by scores: 16 lanes (one DPP row) hold one token.
// Lane i has the experts 64 c + 4 i + q (c < CH, q < 4), so that a row of
// logits is read in whole 128 or 256-byte pieces.
#pragma once

#include "ops_common.h"

namespace moe {
namespace {

constexpr int kTokens = 16;  // per workgroup of 256 lanes
constexpr float kNegInf = -__builtin_inff();

// ---- exchanges within a row of 16 lanes
enum { ROW_XOR1 = 0xB1, ROW_XOR2 = 0x4E, ROW_HALF_MIRROR = 0x141, ROW_MIRROR = 0x140, ROW_NEXT = 0x101 };
// (ROW_NEXT: the next lane's value, 0 in the last)
template <int CTRL>
__device__ __forceinline__ uint32_t row_get(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, CTRL == ROW_NEXT);
}
template <int CTRL>
__device__ __forceinline__ float row_get(float v) {
  return __uint_as_float(row_get<CTRL>(__float_as_uint(v)));
}
template <int CTRL>
__device__ __forceinline__ double row_get(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, (uint64_t)row_get<CTRL>((uint32_t)(b >> 32)) << 32 |
                                        row_get<CTRL>((uint32_t)b));
}
// Lane j of the row's value in all its lanes.
template <int J, class T>
__device__ __forceinline__ T row_lane(T v) {
  return row_get<0x150 + J>(v);
}
// Sums and maxima over a row, the same in every lane: pairs, quads, then the mirrored
// halves, whose lanes agree by then.
template <class T, class F>
__device__ __forceinline__ T row_reduce(T v, F f) {
  v = f(v, row_get<ROW_XOR1>(v));
  v = f(v, row_get<ROW_XOR2>(v));
  v = f(v, row_get<ROW_HALF_MIRROR>(v));
  return f(v, row_get<ROW_MIRROR>(v));
}
template <class T>
__device__ __forceinline__ T row_sum(T v) {
  return row_reduce(v, [](T a, T b) { return a + b; });
}
template <class T>
__device__ __forceinline__ T row_max(T v) {
  return row_reduce(v, [](T a, T b) { return a > b ? a : b; });
}

// Writes to LDS before, reads after: among the lanes of a wavefront (a token has one).
__device__ __forceinline__ void lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// ---- logits of one row; NaN and what lies outside E count as -infinity
__device__ __forceinline__ float usable(float x) { return x == x ? x : kNegInf; }
__device__ __forceinline__ float logit_at(const void* logits, bool bf16, size_t at) {
  return usable(bf16 ? bf16_bits_to_f32(static_cast<const uint16_t*>(logits)[at])
                     : static_cast<const float*>(logits)[at]);
}
template <int CH>
__device__ __forceinline__ void load_logits(const void* logits, bool bf16, size_t row, int E, int i,
                                            float (&x)[4 * CH]) {
  const size_t base = row * E;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int e = 64 * c + 4 * i;
    float* v = x + 4 * c;
    if ((E & 3) == 0) {  // whole vectors: rows start at multiples of 4 values
      v[0] = v[1] = v[2] = v[3] = kNegInf;
      if (e < E) {
        if (bf16) {
          const u32x2 d = *reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(logits) + base + e);
          v[0] = bf16_lo(d[0]), v[1] = bf16_hi(d[0]), v[2] = bf16_lo(d[1]), v[3] = bf16_hi(d[1]);
        } else {
          const f32x4 d = *reinterpret_cast<const f32x4*>(static_cast<const float*>(logits) + base + e);
          v[0] = d[0], v[1] = d[1], v[2] = d[2], v[3] = d[3];
        }
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = usable(v[q]);
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = e + q < E ? logit_at(logits, bf16, base + e + q) : kNegInf;
    }
  }
}

// ---- scores in fp32; errors in half steps, 2^-24 relative
// e^x for x <= 0 as 2^r 2^f, f = x log2 e - r with log2 e in two parts: off by 4 (2 of the
// hardware's power, f's roundings).
__device__ __forceinline__ float exp_neg32(float x) {
  x = fmaxf(x, -200.f);
  const float r = __builtin_rintf(x * 1.44269504f);
  const float f = __builtin_fmaf(x, 1.92596302e-8f, __builtin_fmaf(x, 1.44269504f, -r));
  return __builtin_amdgcn_ldexpf(__builtin_amdgcn_exp2f(f), (int)r);
}
// 1 / (1 + e^-l) from t = e^-|l|: 4 for t, 3 for 1 + t, 2 for its reciprocal, 1 for the product.
__device__ __forceinline__ float sigmoid32(float l) {
  const float t = exp_neg32(-fabsf(l));
  return (l < 0.f ? t : 1.f) * __builtin_amdgcn_rcpf(1.f + t);
}

// ---- scores in fp64, good to a few units of the last place
// e^x for x <= 0: 2^n e^r with |r| <= ln 2 / 2, and the Taylor sum to r^12.
__device__ __forceinline__ double exp_neg(double x) {
  x = x < -800.0 ? -800.0 : x;
  const double n = __builtin_rint(x * 1.4426950408889634074);
  double r = __builtin_fma(n, -0.69314718036912381649, x);  // ln 2 in two parts, the first of 32 bits
  r = __builtin_fma(n, -1.9082149292705877000e-10, r);
  constexpr double c[13] = {1.0,           1.0,            1.0 / 2,         1.0 / 6,         1.0 / 24,
                            1.0 / 120,     1.0 / 720,      1.0 / 5040,      1.0 / 40320,     1.0 / 362880,
                            1.0 / 3628800, 1.0 / 39916800, 1.0 / 479001600};
  double p = c[12];
#pragma unroll
  for (int j = 11; j >= 0; --j) p = __builtin_fma(p, r, c[j]);
  return __builtin_amdgcn_ldexp(p, (int)n);
}
// 1 / d for ordinary d: the hardware's estimate and two steps of Newton's
__device__ __forceinline__ double reciprocal(double d) {
  double y = __builtin_amdgcn_rcp(d);
  y = __builtin_fma(y, __builtin_fma(-d, y, 1.0), y);
  return __builtin_fma(y, __builtin_fma(-d, y, 1.0), y);
}
// s = 1 / (1 + e^-l), from t = e^-|l| <= 1
__device__ __forceinline__ double sigmoid64(double l) {
  const double t = exp_neg(-__builtin_fabs(l));
  return (l < 0.0 ? t : 1.0) * reciprocal(1.0 + t);
}
// a logit in fp64; an infinite one stands for a number that all others vanish next to
constexpr double kHuge = 0x1p996;  // (whose lowest bits are empty)
__device__ __forceinline__ double wide(float x) {
  const double d = (double)x;
  return d > kHuge ? kHuge : d;
}

}  // namespace
}  // namespace moe
