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

// The reciprocal that penalise8 divides by; zero where it must not be used (a
// penalty so far from one that residues would overflow or underflow).
__device__ __forceinline__ float quotient_factor(float repetition) {
  return repetition > 0x1p-100f && repetition < 0x1p100f ? 1.0f / repetition : 0.0f;
}

// Penalty::apply for eight bf16 values whose counts stand in a word of bytes
// (0: not seen, n: n - 1 times among the outputs), without a branch: some of
// them were seen.  The quotient is the product with the rounded reciprocal,
// corrected once by its residue: that is the division to within its last bit
// of fp32 (and almost always to its own rounding), 2^-16 of a step of the bf16
// result.  The fixup puts in what a division gives for infinities, NaN and
// zeros.
__device__ __forceinline__ void penalise8(float (&x)[8], uint64_t n8, const Penalty& p, float inv) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float n = (float)((uint32_t)(n8 >> (8 * i)) & 255u);
    float y = x[i];
    if (p.repeat) {
      const float q = y * inv;
      const float d = __builtin_amdgcn_div_fixupf(__builtin_fmaf(__builtin_fmaf(-q, p.repetition, y), inv, q), p.repetition, y);
      y = y > 0.0f ? d : y * p.repetition;
      y = n > 0.0f ? y : x[i];
    }
    if (p.count) {
      const float off = p.frequency * (n - 1.0f) + p.presence;
      y = n > 1.0f ? y - off : y;
    }
    x[i] = y;
  }
}

// A processed score's order codes (16 bits for bf16 values, 32 for fp32) up to
// these are -inf: nothing was left to draw.
constexpr uint32_t kNothingLeft16 = 0x007Fu;
constexpr uint32_t kNothingLeft32 = 0x007FFFFFu;

}  // namespace dspark
