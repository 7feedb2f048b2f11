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
inline int64_t rule_words(int64_t V) { return V / 32 + (V % 32 != 0); }
struct TableParams {
  RuleSet r;
  uint32_t* seen;
  uint32_t* counts;
  uint64_t* keys;  // of a draft's steps: its first slot is cleared
  int64_t b0;      // first request of a launch (set by the launcher)
  int64_t B;
  int64_t V;
};
hipError_t launch_rule_table(const TableParams& p, hipStream_t s);

// Best keys of a draft's rows: three slots, of steps k = 0, 1, 2 modulo 3,
// each of kStepGroups groups of columns by B rows.  Step k reads the last
// step's slot, meets in its own and clears the next one's; the first step's
// is clear before the draft (launch_rule_table, or a fill).
constexpr int kStepGroups = 8;
constexpr int kStepSlots = 3;

// Step k of a left-to-right draft in one pass: the token of position k - 1
// from its keys, written out and counted; the corrected logits of row (b, k)
// (base plus the bias of that predecessor), the rules, the processed row to
// `out`, and the row's best keys.
struct RuleStepParams {
  RuleSet r;
  const void* base;        // [B, M, V]
  void* out;               // [B, M, V]
  const int64_t* first;    // [B] predecessors of position 0
  int64_t* tokens;         // [B, M]
  const void* w1;          // [V, rank]
  const void* w2;          // [V, rank]
  uint32_t* seen;          // table, or null (no penalty)
  uint32_t* counts;        // readable 256 bytes past its end
  uint64_t* keys;          // [kStepSlots][kStepGroups][B]
  uint32_t* bad_rows;
  int64_t b0;              // first row of a launch (set by the launcher)
  int64_t B;
  int64_t M;
  int64_t V;
  int64_t rank;
  int64_t k;
  int64_t batch_offset;
  float kappa;             // (float)(log2(e) / T), above zero; unused when greedy
  uint32_t k_abs;
  uint32_t seed_lo;
  uint32_t seed_hi;
  bool greedy;
};
hipError_t launch_rule_step(const RuleStepParams& p, bool logits_bf16, bool weights_bf16, int num_cus, hipStream_t s);

// tokens[b, M - 1] = the column of the row's best key, -1 when it has none.
hipError_t launch_rule_choose(const uint64_t* keys, int64_t B, int64_t M, int64_t* tokens, hipStream_t s);

}  // namespace dspark
