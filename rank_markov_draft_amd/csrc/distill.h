// distill.h -- interface of the distillation loss (distill.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dspark {

// Entries of a teacher's list.
constexpr int64_t kDistillMaxEntries = 1024;

struct DistillParams {
  const void* logits;           // [rows, V]
  const int64_t* teacher_ids;   // [rows, K]
  const void* teacher_logits;   // [rows, K]
  float* loss;                  // [rows]
  float* stats;                 // [rows, 4]: the row's largest logit and the sum of its weights, the teacher's likewise
  float* partials;              // [rows, slices, 2] largest logit and sum of a slice; unused with one slice
  const float* grad_loss;       // [rows], backward
  void* grad;                   // [rows, V], backward; may be logits
  int64_t rows;
  int64_t V;
  int64_t K;
  double tau;
  float kappa;                  // log2(e) / tau
  bool teacher_bf16;
};

// Slices that the forward pass cuts a row into.
int64_t distill_slices(int64_t rows, int64_t V);

hipError_t launch_distill_loss(const DistillParams& p, bool bf16, hipStream_t s);
hipError_t launch_distill_backward(const DistillParams& p, bool bf16, hipStream_t s);

}  // namespace dspark
