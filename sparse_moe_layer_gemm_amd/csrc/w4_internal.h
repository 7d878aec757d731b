// Declarations of 4-bit integer weights with group scales (internal).
#pragma once

#include "ops_internal.h"

namespace moe {

// A format: groups of `group` values along K share a scale (bf16 or fp32) and,
// where zeros is not null, a zero point (else 8): w = (q - z) * s.
struct W4 {
  const uint8_t* codes;  // two codes a byte, the even one low
  const void* scales;
  const uint8_t* zeros;
  bool scale_f32;
  int group;
};

hipError_t launch_w4_quantize_rows(const void* x, bool bf16, long long R, int K, int group, uint8_t* codes,
                                   bool scale_f32, void* scales, uint8_t* zeros, hipStream_t st);
hipError_t launch_w4_quantize_cols(const void* x, bool bf16, long long B, int K, int C, int group,
                                   uint8_t* codes, bool scale_f32, void* scales, uint8_t* zeros,
                                   hipStream_t st);
hipError_t launch_w4_dequantize(const W4& w, long long R, int K, bool bf16, void* out, hipStream_t st);

// Products of bf16 rows (g.a; g.w and g.w_scale are not used) with such weights [E, N, K]: streamed, for experts
// with few rows, or on tiles.
hipError_t launch_w4_stream(const GroupedArgs& g, const W4& w, hipStream_t st);
hipError_t launch_w4_tile(const GroupedArgs& g, const W4& w, hipStream_t st);
bool w4_prefer_stream(const GroupedArgs& g, const W4& w);

}  // namespace moe
