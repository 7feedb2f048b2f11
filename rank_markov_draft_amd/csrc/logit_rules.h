// logit_rules.h -- interface of the logit rules (logit_rules.hip): penalties
// for repeated tokens, biases and grammar masks on corrected logits.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dspark {

// The rules of a call, as dspark_logit_rules_t holds them (device pointers;
// null: that rule is off).
struct RuleSet {
  const int64_t* history;         // [B] rows of history_len ids, history_stride apart
  const int64_t* lengths;         // [B] ids of each row that count, or null: all
  const int64_t* prompt_lengths;  // [B] ids of those that are the prompt's, or null: none
  const float* repetition;        // [B]
  const float* frequency;         // [B]
  const float* presence;          // [B]
  const void* bias;               // rows of V biases, bias_stride elements apart (0: one row)
  const uint32_t* mask;           // packed allowed bits, word strides below (0: shared)
  int64_t history_len;
  int64_t history_stride;
  int64_t bias_stride;
  int64_t mask_stride_b;
  int64_t mask_stride_m;
  bool bias_bf16;
};

// Whether any penalty is on, so that the tokens have to be counted.
inline bool rules_penalise(const RuleSet& r) {
  return r.repetition != nullptr || r.frequency != nullptr || r.presence != nullptr;
}

// The rules on given logits (grad null), or the gradient with respect to the
// logits (grad set: out = grad times the rules' slope).
struct RulesParams {
  RuleSet r;
  const void* logits;        // [B, M, V]
  const void* grad;          // [B, M, V] or null
  void* out;                 // [B, M, V]; may be logits (or grad)
  const int64_t* token_ids;  // [B, M] or null
  int64_t B;
  int64_t M;
  int64_t V;
};
hipError_t launch_logit_rules(const RulesParams& p, bool logits_bf16, int num_cus, hipStream_t s);

// The tokens of each row's history as a table: a bit per token that stands in
// it (rule_words(V) words a row), and its count among the outputs where the
// bit is set (V words a row; other counts are left unwritten).
inline int64_t rule_words(int64_t V) { return (V + 31) / 32; }
struct TableParams {
  RuleSet r;
  uint32_t* seen;
  uint32_t* counts;
  int64_t B;
  int64_t V;
};
hipError_t launch_rule_table(const TableParams& p, hipStream_t s);

// Step k of a left-to-right draft in one pass: the corrected logits of row
// (b, k) (base plus the bias of its predecessor), the rules, the processed row
// to `out`, and the row's best keys over rule_step_parts(V) blocks of columns.
struct RuleStepParams {
  RuleSet r;
  const void* base;        // [B, M, V]
  void* out;               // [B, M, V]
  const int64_t* first;    // [B] predecessors of position 0
  const int64_t* tokens;   // [B, M] predecessors of the others, at k - 1
  const void* w1;          // [V, rank]
  const void* w2;          // [V, rank]
  const uint32_t* seen;    // table, or null (no penalty)
  const uint32_t* counts;  // readable 256 bytes past its end
  uint64_t* partials;      // [B, rule_step_parts(V)]: read by launch_rule_choose (keys null)
  // or: the last workgroup of a row chunk to finish draws its tokens itself.
  // Zero before the launch, left zero.
  uint64_t* keys;          // [B]
  uint32_t* arrived;       // one word (keys: B at most 16)
  int64_t* tokens_out;     // [B, M] (the same as tokens)
  uint32_t* seen_out;      // (the same as seen)
  uint32_t* counts_out;    // (the same as counts)
  uint32_t* bad_rows;
  int64_t B;
  int64_t M;
  int64_t V;
  int64_t rank;
  int64_t k;
  int64_t batch_offset;
  float kappa;             // (float)(log2(e) / T); unused when greedy
  uint32_t k_abs;
  uint32_t seed_lo;
  uint32_t seed_hi;
  bool greedy;
};
int64_t rule_step_parts(int64_t V);
hipError_t launch_rule_step(const RuleStepParams& p, bool logits_bf16, bool weights_bf16, hipStream_t s);

// tokens[b, k] = the column of the row's best key, -1 when its score is -inf;
// a drawn token joins the table (seen null: no table).
hipError_t launch_rule_choose(const uint64_t* partials, int64_t nparts, int64_t B, int64_t M, int64_t k, int64_t V,
                              int64_t* tokens, uint32_t* seen, uint32_t* counts, hipStream_t s);

}  // namespace dspark
