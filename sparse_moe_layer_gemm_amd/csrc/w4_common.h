// Device pieces of the products with 4-bit integer weights.
#pragma once

#include "grouped_common.h"
#include "w4_internal.h"

namespace moe {
namespace {

// 8 codes (one dword, element 2j in the low nibble of byte j) -> their values 0 .. 15 as
// bf16, in the order 0 2 4 6 1 3 5 7: a byte 0 .. 15 read as E4M3 is the code times 2^-9
// (subnormal up to 7, the first binade from 8), and the converter takes a power of two.
__device__ __forceinline__ u32x4 code_frag(uint32_t d) {
  const int even = (int)(d & 0x0F0F0F0Fu), odd = (int)((d >> 4) & 0x0F0F0F0Fu);
  u32x4 r;
  r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(even, 512.f, false));
  r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(even, 512.f, true));
  r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(odd, 512.f, false));
  r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(odd, 512.f, true));
  return r;
}
// Four codes, a byte each, as two pairs of bf16.
__device__ __forceinline__ void code_pairs(u32x4& r, uint32_t bytes, int at) {
  r[at] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)bytes, 512.f, false));
  r[at + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)bytes, 512.f, true));
}
// The same as code_frag in the codes' own order.
__device__ __forceinline__ u32x4 code_frag_in_order(uint32_t d) {
  const uint32_t even = d & 0x0F0F0F0Fu, odd = (d >> 4) & 0x0F0F0F0Fu;
  u32x4 r;
  code_pairs(r, __builtin_amdgcn_perm(odd, even, 0x05010400u), 0);
  code_pairs(r, __builtin_amdgcn_perm(odd, even, 0x07030602u), 2);
  return r;
}
// 8 adjacent bf16 in the order of code_frag
__device__ __forceinline__ u32x4 row_frag(const u32x4& x) {
  u32x4 r;
  r[0] = __builtin_amdgcn_perm(x[1], x[0], 0x05040100u);
  r[1] = __builtin_amdgcn_perm(x[3], x[2], 0x05040100u);
  r[2] = __builtin_amdgcn_perm(x[1], x[0], 0x07060302u);
  r[3] = __builtin_amdgcn_perm(x[3], x[2], 0x07060302u);
  return r;
}
__device__ __forceinline__ f32x4 mfma16(const u32x4& a, const u32x4& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

}  // namespace
}  // namespace moe
