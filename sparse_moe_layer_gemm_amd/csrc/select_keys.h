// The 32-bit keys of routing by scores, in plain C++ (constexpr functions are for host and device).
#pragma once

#include <stdint.h>

namespace moe {

// Key of expert e, whose choice c stands at `units` in the range that 24 bits hold: below 1 counts as 1 (and so does
// a NaN, of two infinite choices), and 2^24 - 1 is the largest. What is left out (c = -infinity) has 0 there. The
// conversion to a whole number is of a number between 0 and 2^24 always: of others it is undefined.
constexpr uint32_t choice_key(float c, float units, int e) {
  const float at = c == -__builtin_inff() ? 0.f : __builtin_fmaxf(units, 1.f);
  return (uint32_t)at << 8 | (uint32_t)(255 - e);
}

}  // namespace moe
