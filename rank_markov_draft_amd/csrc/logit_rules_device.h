// logit_rules_device.h -- the penalties of the logit rules, as the kernels
// apply them (logit_rules.hip, and the greedy chain in markov_chain.hip).
#pragma once

#include "device_common.h"
#include "logit_rules.h"

namespace dspark {

// A request's penalties; a rule that is off leaves x as it is.
struct Penalty {
  float repetition, frequency, presence;
  bool repeat, count;
  __device__ __forceinline__ float apply(float x, uint32_t c) const {
    if (repeat) x = x > 0.0f ? x / repetition : x * repetition;
    if (count && c > 0u) x = x - (frequency * (float)c + presence);
    return x;
  }
};
__device__ __forceinline__ Penalty penalty_of(const RuleSet& r, int64_t b) {
  return Penalty{r.repetition ? r.repetition[b] : 1.0f, r.frequency ? r.frequency[b] : 0.0f,
                 r.presence ? r.presence[b] : 0.0f, r.repetition != nullptr,
                 r.frequency != nullptr || r.presence != nullptr};
}

// A processed score's order codes (16 bits for bf16 values, 32 for fp32) up to
// these are -inf: nothing was left to draw.
constexpr uint32_t kNothingLeft16 = 0x007Fu;
constexpr uint32_t kNothingLeft32 = 0x007FFFFFu;

}  // namespace dspark
