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

// The quotient of a bf16 value y and a penalty from the penalty's reciprocal in
// two words: y * high + y * low with one rounding at the end.  That is the
// division's own rounding for all 2^30 pairs of significands of y and of the
// penalty but two, whose penalties are left out.  Where no step leaves the
// normal range it does not depend on the exponents either: penalties within
// 2^-20 .. 2^20, and values that are zero or within 2^-50 .. 2^100, so that
// quotients stay below 2^120, the products with the low word above 2^-126, and
// neither infinities nor NaN come up.  Others are divided.
struct Reciprocal {
  float high, low;  // high: zero for a penalty to divide by
};
__device__ __forceinline__ Reciprocal reciprocal_of(float repetition) {
  const uint32_t s = __float_as_uint(repetition) & 0x7FFFFFu;
  if (!(repetition >= 0x1p-20f && repetition <= 0x1p20f) || s == 0x50AB43u || s == 0x792863u) return {0.0f, 0.0f};
  const float high = 1.0f / repetition;
  return {high, __builtin_fmaf(-repetition, high, 1.0f) / repetition};
}

// Whether all of eight packed bf16 values are in that range.
__device__ __forceinline__ bool plain_dividends(const uint32_t (&w)[4]) {
  typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
  constexpr uint32_t kLow = (127 - 50) << 7, kHigh = (127 + 100) << 7;
  u16x2_t low = {0xFFFF, 0xFFFF}, high = {0, 0};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const u16x2_t m = __builtin_bit_cast(u16x2_t, w[q] & 0x7FFF7FFFu);
    low = __builtin_elementwise_min(low, (u16x2_t)(m - (uint16_t)1));  // zeros come last
    high = __builtin_elementwise_max(high, m);
  }
  return min((uint32_t)low[0], (uint32_t)low[1]) >= kLow - 1 && max((uint32_t)high[0], (uint32_t)high[1]) <= kHigh;
}

// Penalty::apply for eight bf16 values whose counts stand in a word of bytes
// (0: not seen, n: n - 1 times among the outputs), without a branch: some of
// them were seen.  For plain_dividends, and a reciprocal that is not zero.
__device__ __forceinline__ void penalise8(float (&x)[8], uint64_t n8, const Penalty& p, const Reciprocal& r) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float n = (float)((uint32_t)(n8 >> (8 * i)) & 255u);
    float y = x[i];
    if (p.repeat) {
      y = y > 0.0f ? __builtin_fmaf(y, r.high, y * r.low) : y * p.repetition;
      y = n > 0.0f ? y : x[i];
    }
    if (p.count) {
      const float off = p.frequency * (n - 1.0f) + p.presence;
      y = n > 1.0f ? y - off : y;
    }
    x[i] = y;
  }
}

// The greedy chain's order codes (16 bits) up to this are -inf: nothing was
// left to draw.
constexpr uint32_t kNothingLeft16 = 0x007Fu;

}  // namespace dspark
