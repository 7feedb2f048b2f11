// token_filter.h -- interface of sampling under a request's limits
// (token_filter.hip): temperature, top-k, top-p and min-p.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dspark {

// A limit of every request, or one for all where the pointer is null.
struct TokenLimits {
  const float* temperature;
  const int64_t* top_k;
  const float* top_p;
  const float* min_p;
  int64_t all_top_k;
  float all_temperature;
  float all_top_p;
  float all_min_p;
};

constexpr int kFilterGroup = 128;  // columns of a group
struct FilterParams {
  TokenLimits limits;
  const void* logits;     // [B, M, V]
  const float* uniforms;  // [B, M]
  int64_t* tokens;        // [B, M]
  float* probs;           // [B, M]
  double* sums;           // [rows, filter_groups(V)] sums of a group's weights, of rows that need them
  uint32_t* tops;         // [rows, filter_groups(V)] order codes of the groups' largest logits
  int64_t rows;
  int64_t M;
  int64_t V;
};
__host__ __device__ inline int64_t filter_groups(int64_t V) { return (V + kFilterGroup - 1) / kFilterGroup; }

hipError_t launch_token_filter(const FilterParams& p, bool bf16, hipStream_t s);

}  // namespace dspark
