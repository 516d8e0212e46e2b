// The rule of a grouped routing call, and its logits.
#pragma once

#include "moe_common.h"

namespace moe {
namespace {

struct RouteRule {
  int T, E, k;
  int groups, kept, group_top;
  bool renormalise, softmax, bf16;
  float scale;
};

// Lanes of a group: 64 shared out over the groups, rounded up to a power of
// two; each lane holds at most kMaxPerLane of its group's experts.
constexpr int kMaxPerLane = 16;
inline int group_lanes(int groups) {
  int l = kWave;
  while (l > 1 && l * groups > kWave) l >>= 1;
  return l;
}

// A logit or bias at or below this, or NaN, masks its expert: -inf and the
// lowest finite value of fp32 and of bf16 (-3.39e38) alike.
constexpr float kLowest = -3.3e38f;

// Logit i in 64 bits; masked ones as -inf, +inf as the largest float (so that
// a softmax over it is defined: such experts share all of the weight).
__device__ __forceinline__ double load_logit(const void* __restrict__ p, bool bf16, size_t i) {
  const float z = bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16)
                       : static_cast<const float*>(p)[i];
  return z > kLowest ? (double)fminf(z, 3.402823466e+38f) : -__builtin_huge_val();
}

}  // namespace
}  // namespace moe
