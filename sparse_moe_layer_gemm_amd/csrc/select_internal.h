// Declarations of routing by scores (internal).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

struct SelectArgs {
  const void* logits;  // [T, E]
  bool bf16, sigmoid, renorm;
  int T, E, k;
  const float* bias;  // [E], or null
  int groups, group_k, group_top;
  int group_size, group_magic, lds_stride;  // set by the launch
  float scale;
  int32_t* ids;  // [T, k]
  float* w;      // [T, k]
  float* scores;  // [T, E], or null
};
hipError_t launch_select(SelectArgs a, hipStream_t st);

struct SelectGradArgs {
  const void* logits;  // [T, E]
  bool bf16, sigmoid, renorm, dl_bf16;
  int T, E, k;
  float scale;
  const int32_t* ids;    // [T, k]
  const float* dw;       // [T, k]
  const float* dscores;  // [T, E], or null
  void* dl;              // [T, E]
};
hipError_t launch_select_backward(const SelectGradArgs& a, hipStream_t st);

}  // namespace moe
