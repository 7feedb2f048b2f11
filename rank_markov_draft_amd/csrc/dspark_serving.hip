// dspark_serving.hip -- host side of the 8-bit vocabulary head and of the
// logit rules (include/dspark_markov.h): argument validation, workspace
// layout and launches.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstring>

#include "dspark_markov.h"
#include "host_common.h"
#include "int8_head.h"
#include "logit_rules.h"
#include "markov_kernels.h"

namespace {

using namespace dspark::host;

int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// ---- 8-bit head: the quantised rows, then their scales and the floats past
// them that the product reads in whole vectors
size_t int8_rows_bytes(int64_t rows, int64_t d) {
  return align256(mul_sz((size_t)rows, (size_t)round_up(d, dspark::kInt8K)));
}
size_t int8_scales_bytes(int64_t rows) {
  return align256(mul_sz(add_sz((size_t)rows, (size_t)dspark::kInt8RowPad), sizeof(float)));
}

// ---- logit rules
// Byte ranges that a call's rules read, for the overlap checks.
struct Ranges {
  const void* at[16];
  size_t bytes[16];
  int n = 0;
  void add(const void* p, size_t b) {
    at[n] = p;
    bytes[n++] = b;
  }
  bool meet(const void* p, size_t b) const {
    for (int i = 0; i < n; ++i)
      if (overlaps(p, b, at[i], bytes[i])) return true;
    return false;
  }
};

// Bytes from the first to the last element of `count` rows of `len` elements
// `stride` apart; -1 when they cannot be represented.
int64_t extent(int64_t count, int64_t stride, int64_t len, int64_t size) {
  int64_t t = 0;
  if (count <= 0 || len <= 0) return 0;
  if (!mul_ok(count - 1, stride, &t) || __builtin_add_overflow(t, len, &t) || !mul_ok(t, size, &t)) return -1;
  return t;
}

dspark_status_t check_rules(const dspark_logit_rules_t* c, int64_t B, int64_t M, int64_t V, dspark::RuleSet* r,
                            Ranges* in, int64_t* mask_bytes) {
  if (!c) return DSPARK_ERR_INVALID_ARGUMENT;
  if (c->history && (c->history_len < 0 || (B > 1 && c->history_stride < c->history_len)))
    return DSPARK_ERR_INVALID_ARGUMENT;
  if (c->logit_bias && (!known_dtype(c->bias_dtype) || (c->bias_stride != 0 && c->bias_stride < V)))
    return DSPARK_ERR_INVALID_ARGUMENT;
  if (c->token_mask && (c->mask_stride_b < 0 || c->mask_stride_m < 0)) return DSPARK_ERR_INVALID_ARGUMENT;
  const int64_t W = dspark::rule_words(V);
  const size_t vec = (size_t)B * sizeof(float), ids = (size_t)B * sizeof(int64_t);
  int64_t hist = 0, bias = 0, mask = 0, mm = 0;
  if (c->history && c->history_len > 0) hist = extent(B, B > 1 ? c->history_stride : 0, c->history_len, 8);
  if (c->logit_bias) bias = extent(B, c->bias_stride, V, (int64_t)dtype_bytes(c->bias_dtype));
  if (c->token_mask) {
    if (!mul_ok(M - 1, c->mask_stride_m, &mm) || __builtin_add_overflow(mm, W, &mm)) return DSPARK_ERR_INVALID_ARGUMENT;
    mask = extent(B, c->mask_stride_b, mm, 4);
  }
  if (hist < 0 || bias < 0 || mask < 0) return DSPARK_ERR_INVALID_ARGUMENT;
  in->add(c->history, (size_t)hist);
  in->add(c->history ? c->lengths : nullptr, ids);
  in->add(c->history ? c->prompt_lengths : nullptr, ids);
  in->add(c->repetition_penalty, vec);
  in->add(c->frequency_penalty, vec);
  in->add(c->presence_penalty, vec);
  in->add(c->logit_bias, (size_t)bias);
  in->add(c->token_mask, (size_t)mask);
  *mask_bytes = mask;
  *r = dspark::RuleSet{};
  if (c->history && c->history_len > 0) {
    r->history = c->history;
    r->lengths = c->lengths;
    r->prompt_lengths = c->prompt_lengths;
    r->history_len = c->history_len;
    r->history_stride = B > 1 ? c->history_stride : 0;
  }
  r->repetition = c->repetition_penalty;
  r->frequency = c->frequency_penalty;
  r->presence = c->presence_penalty;
  r->bias = c->logit_bias;
  r->bias_stride = c->bias_stride;
  r->bias_bf16 = c->logit_bias && c->bias_dtype == DSPARK_BF16;
  r->mask = c->token_mask;
  r->mask_stride_b = c->mask_stride_b;
  r->mask_stride_m = c->mask_stride_m;
  return DSPARK_OK;
}

// The rules on logits, or their gradient (grad not null).
dspark_status_t run_rules(const void* grad, const void* logits, dspark_dtype_t dtype, const int64_t* token_ids,
                          const dspark_logit_rules_t* rules, int64_t B, int64_t M, int64_t V, void* out, bool backward,
                          void* stream) {
  if (!known_dtype(dtype) || B < 0 || M < 0 || V < 0) return DSPARK_ERR_INVALID_ARGUMENT;
  int64_t rows = 0, elems = 0, bytes = 0;
  if (!mul_ok(B, M, &rows) || !mul_ok(rows, V, &elems) || !mul_ok(elems, 4, &bytes)) return DSPARK_ERR_INVALID_ARGUMENT;
  if (V > ((int64_t)1 << 30)) return DSPARK_ERR_UNSUPPORTED;
  if (!rules) return DSPARK_ERR_INVALID_ARGUMENT;
  if (elems == 0) return DSPARK_OK;
  dspark::RulesParams p{};
  Ranges in;
  int64_t mask_bytes = 0;
  const dspark_status_t st = check_rules(rules, B, M, V, &p.r, &in, &mask_bytes);
  if (st != DSPARK_OK) return st;
  if (!logits || !out || (backward && !grad)) return DSPARK_ERR_INVALID_ARGUMENT;
  const size_t lbytes = (size_t)elems * dtype_bytes(dtype);
  in.add(token_ids, (size_t)rows * sizeof(int64_t));
  const void* const streamed = backward ? grad : logits;
  if (out != streamed && overlaps(out, lbytes, streamed, lbytes)) return DSPARK_ERR_INVALID_ARGUMENT;
  if (backward && overlaps(out, lbytes, logits, lbytes)) return DSPARK_ERR_INVALID_ARGUMENT;
  if (in.meet(out, lbytes)) return DSPARK_ERR_INVALID_ARGUMENT;
  if (backward) p.r.bias = nullptr;
  p.logits = logits;
  p.grad = grad;
  p.out = out;
  p.token_ids = token_ids;
  p.B = B;
  p.M = M;
  p.V = V;
  const int cus = device_cus();
  const hipError_t e = dspark::launch_logit_rules(p, dtype == DSPARK_BF16, cus > 0 ? cus : 1, (hipStream_t)stream);
  if (e == hipErrorNotSupported) {
    (void)hipGetLastError();
    return DSPARK_ERR_UNSUPPORTED;
  }
  if (e != hipSuccess) return device_failure(e, "logit rules launch");
  return DSPARK_OK;
}

// Workspace of a processed draft past the vanilla sampling layout: the table's
// bits, its counts, and the steps' keys.
size_t table_bits_bytes(int64_t B, int64_t V) {
  return align256(mul_sz(mul_sz((size_t)B, (size_t)dspark::rule_words(V)), 4));
}
size_t table_counts_bytes(int64_t B, int64_t V) {
  return align256(add_sz(mul_sz(mul_sz((size_t)B, (size_t)V), 4), 256));  // read in whole groups of 64 columns
}
size_t step_keys_bytes(int64_t B) { return align256(mul_sz((size_t)B, dspark::kStepSlots * dspark::kStepGroups * sizeof(uint64_t))); }

}  // namespace

extern "C" {

dspark_status_t dspark_markov_quantize_rows(const void* x, dspark_dtype_t dtype, int64_t rows, int64_t d, int8_t* q,
                                            float* scale, void* stream) {
  if (!known_dtype(dtype) || rows < 0 || d < 0) return DSPARK_ERR_INVALID_ARGUMENT;
  int64_t n = 0, bytes = 0;
  if (!mul_ok(rows, d, &n) || !mul_ok(n, 4, &bytes) || !mul_ok(rows, 4, &bytes)) return DSPARK_ERR_INVALID_ARGUMENT;
  if (rows > (int64_t)0x7FFFFFFF) return DSPARK_ERR_UNSUPPORTED;
  if (rows == 0) return DSPARK_OK;
  if (!scale || (d > 0 && (!x || !q))) return DSPARK_ERR_INVALID_ARGUMENT;
  const size_t xb = (size_t)n * dtype_bytes(dtype), sb = (size_t)rows * sizeof(float);
  if (overlaps(q, (size_t)n, x, xb) || overlaps(scale, sb, x, xb) || overlaps(q, (size_t)n, scale, sb))
    return DSPARK_ERR_INVALID_ARGUMENT;
  const hipStream_t s = (hipStream_t)stream;
  const dspark::QuantizeParams p{x, q, scale, rows, d, d};
  const hipError_t e = d == 0 ? dspark::launch_fill_zero(scale, sb, s) : dspark::launch_quantize_rows(p, dtype == DSPARK_BF16, s);
  if (e != hipSuccess) return device_failure(e, "quantize launch");
  return DSPARK_OK;
}

size_t dspark_markov_lm_head_int8_workspace_bytes(int64_t B, int64_t M, int64_t d) {
  if (B < 0 || M < 0 || d < 0 || d > dspark::kInt8MaxInner) return kDataOffset;
  int64_t rows = 0;
  if (!mul_ok(B, M, &rows)) return SIZE_MAX;
  return add_sz(kDataOffset, add_sz(int8_rows_bytes(rows, d), int8_scales_bytes(rows)));
}

dspark_status_t dspark_markov_lm_head_int8(const void* hidden_states, dspark_dtype_t hidden_dtype, int64_t d,
                                           const int8_t* head_q, const float* head_scale, int64_t B, int64_t M,
                                           int64_t V, void* logits, dspark_dtype_t logits_dtype, void* workspace,
                                           size_t workspace_bytes, void* stream) {
  if (!known_dtype(hidden_dtype) || !known_dtype(logits_dtype)) return DSPARK_ERR_INVALID_ARGUMENT;
  if (B < 0 || M < 0 || V < 0 || d <= 0) return DSPARK_ERR_INVALID_ARGUMENT;
  int64_t rows = 0, elems = 0, t = 0;
  if (!mul_ok(B, M, &rows) || !mul_ok(rows, V, &elems) || !mul_ok(elems, 4, &t) || !mul_ok(V, d, &t) ||
      !mul_ok(rows, d, &t) || !mul_ok(t, 4, &t))
    return DSPARK_ERR_INVALID_ARGUMENT;
  if (d > dspark::kInt8MaxInner) {
    dspark::set_last_error("lm_head_int8: the hidden size must be at most 131072");
    return DSPARK_ERR_UNSUPPORTED;
  }
  if (rows > (int64_t)0x7FFFFFFF || V > (int64_t)0x7FFFFFFF) return DSPARK_ERR_UNSUPPORTED;
  if (elems == 0) return DSPARK_OK;
  if (!hidden_states || !head_q || !head_scale || !logits) return DSPARK_ERR_INVALID_ARGUMENT;
  if (!workspace || workspace_bytes < dspark_markov_lm_head_int8_workspace_bytes(B, M, d))
    return DSPARK_ERR_WORKSPACE_TOO_SMALL;
  const size_t obytes = (size_t)elems * dtype_bytes(logits_dtype);
  Ranges in;
  in.add(hidden_states, (size_t)(rows * d) * dtype_bytes(hidden_dtype));
  in.add(head_q, (size_t)(V * d));
  in.add(head_scale, (size_t)V * sizeof(float));
  if (in.meet(logits, obytes)) return DSPARK_ERR_INVALID_ARGUMENT;
  const hipStream_t s = (hipStream_t)stream;
  dspark::Int8HeadParams p{};
  int8_t* const xq = (int8_t*)workspace + kDataOffset;
  float* const xs = (float*)(xq + int8_rows_bytes(rows, d));
  p.xq = xq;
  p.xs = xs;
  p.wq = head_q;
  p.ws = head_scale;
  p.out = logits;
  p.rows = rows;
  p.V = V;
  p.d = d;
  p.ldx = round_up(d, dspark::kInt8K);
  const dspark::QuantizeParams q{hidden_states, xq, xs, rows, d, p.ldx};
  hipError_t e = dspark::launch_quantize_rows(q, hidden_dtype == DSPARK_BF16, s);
  if (e != hipSuccess) return device_failure(e, "hidden state quantize launch");
  e = dspark::launch_int8_head(p, logits_dtype == DSPARK_BF16, device_cus(), s);
  if (e == hipErrorNotSupported) {
    (void)hipGetLastError();
    return DSPARK_ERR_UNSUPPORTED;
  }
  if (e != hipSuccess) return device_failure(e, "int8 head launch");
  return DSPARK_OK;
}

dspark_status_t dspark_markov_process_block(const void* logits, dspark_dtype_t logits_dtype, const int64_t* token_ids,
                                            const dspark_logit_rules_t* rules, int64_t B, int64_t M, int64_t V,
                                            void* processed, void* stream) {
  return run_rules(nullptr, logits, logits_dtype, token_ids, rules, B, M, V, processed, false, stream);
}

dspark_status_t dspark_markov_process_block_backward(const void* grad_processed, const void* logits,
                                                     dspark_dtype_t logits_dtype, const int64_t* token_ids,
                                                     const dspark_logit_rules_t* rules, int64_t B, int64_t M, int64_t V,
                                                     void* grad_logits, void* stream) {
  // only the repetition penalty has a slope: the others shift
  dspark_logit_rules_t slope{};
  if (rules) {
    slope = *rules;
    slope.frequency_penalty = slope.presence_penalty = nullptr;
  }
  return run_rules(grad_processed, logits, logits_dtype, token_ids, rules ? &slope : nullptr, B, M, V, grad_logits, true,
                   stream);
}

size_t dspark_markov_processed_workspace_bytes(int64_t B, int64_t M, int64_t V, int64_t r) {
  const size_t base = align256(dspark_markov_workspace_bytes(B, M, V, r, 1));
  if (B < 0 || M < 0 || V < 0) return base;
  return add_sz(base, add_sz(step_keys_bytes(B), add_sz(table_bits_bytes(B, V), table_counts_bytes(B, V))));
}

dspark_status_t dspark_markov_sample_block_processed(const void* base_logits, dspark_dtype_t logits_dtype,
                                                     const int64_t* first_prev_token_ids, const void* w1,
                                                     const void* w2, dspark_dtype_t weight_dtype,
                                                     const dspark_logit_rules_t* rules, int64_t B, int64_t M,
                                                     int64_t V, int64_t r, double temperature, uint64_t seed,
                                                     int64_t position_offset, int64_t batch_offset,
                                                     int64_t* sampled_tokens, void* processed_logits, void* workspace,
                                                     size_t workspace_bytes, void* stream) {
  int64_t elems = 0;
  dspark_status_t st = check_common(logits_dtype, weight_dtype, B, M, V, r, &elems);
  if (st != DSPARK_OK) return st;
  if (std::isnan(temperature) || !rules) return DSPARK_ERR_INVALID_ARGUMENT;
  if (V > ((int64_t)1 << 30) || r > kGenericMaxRank) return DSPARK_ERR_UNSUPPORTED;
  if (B == 0 || M == 0) return DSPARK_OK;
  if (V == 0) return DSPARK_ERR_INVALID_ARGUMENT;  // nothing to draw from
  dspark::RuleStepParams p{};
  Ranges in;
  int64_t mask_bytes = 0;
  st = check_rules(rules, B, M, V, &p.r, &in, &mask_bytes);
  if (st != DSPARK_OK) return st;
  if (!base_logits || !first_prev_token_ids || !w1 || !w2 || !sampled_tokens || !processed_logits)
    return DSPARK_ERR_INVALID_ARGUMENT;
  if (!workspace || workspace_bytes < dspark_markov_processed_workspace_bytes(B, M, V, r))
    return DSPARK_ERR_WORKSPACE_TOO_SMALL;
  const size_t lbytes = (size_t)elems * dtype_bytes(logits_dtype);
  const size_t wbytes = (size_t)(V * r) * dtype_bytes(weight_dtype);
  const size_t tbytes = (size_t)(B * M) * sizeof(int64_t);
  in.add(base_logits, lbytes);
  in.add(w1, wbytes);
  in.add(w2, wbytes);
  in.add(first_prev_token_ids, (size_t)B * sizeof(int64_t));
  if (in.meet(sampled_tokens, tbytes) || in.meet(processed_logits, lbytes) ||
      overlaps(processed_logits, lbytes, sampled_tokens, tbytes))
    return DSPARK_ERR_INVALID_ARGUMENT;

  const hipStream_t s = (hipStream_t)stream;
  char* const region = (char*)workspace + align256(dspark_markov_workspace_bytes(B, M, V, r, 1));
  uint32_t* const seen = (uint32_t*)region;
  uint32_t* const counts = (uint32_t*)(region + table_bits_bytes(B, V));
  uint64_t* const keys = (uint64_t*)((char*)counts + table_counts_bytes(B, V));
  // without penalties, or with nothing before a single position, no token is
  // ever looked up
  const bool table = dspark::rules_penalise(p.r) && (p.r.history != nullptr || M > 1);
  hipError_t e = hipSuccess;
  if (table) {
    dspark::TableParams t{};
    t.r = p.r;
    t.seen = seen;
    t.counts = counts;
    t.keys = keys;
    t.B = B;
    t.V = V;
    e = dspark::launch_rule_table(t, s);
    if (e != hipSuccess) return device_failure(e, "rule table launch");
  }
  p.base = base_logits;
  p.out = processed_logits;
  p.first = first_prev_token_ids;
  p.tokens = sampled_tokens;
  p.w1 = w1;
  p.w2 = w2;
  p.seen = table ? seen : nullptr;
  p.counts = counts;
  p.keys = keys;
  p.bad_rows = &((Control*)workspace)->bad_rows;
  p.B = B;
  p.M = M;
  p.V = V;
  p.rank = r;
  p.batch_offset = batch_offset;
  p.greedy = temperature < 1e-5;
  // above zero at any temperature, so that an infinite logit's score is not NaN
  p.kappa = p.greedy ? 0.0f : std::fmax((float)(1.4426950408889634 / temperature), 0x1p-149f);
  p.seed_lo = (uint32_t)(seed & 0xFFFFFFFFu);
  p.seed_hi = (uint32_t)(seed >> 32);
  // Greedy drafts with bf16 logits and weights that the persistent chain can
  // hold run as one launch (per-request biases do not fit in its LDS).  The
  // rows and tokens are the steps' own either way.  Whole calls in us, drafts
  // of five by the chain and by steps (and single positions), with penalties
  // and masks: V = 129280 at rank 256, 4 rows 57, 83 (29, 21), 16 rows 68, 99
  // (32, 25), 64 rows 107, 206 (48, 46); V = 32000 at rank 256, 4 rows 44, 50
  // (22, 19), 64 rows 69, 96 (30, 24); at rank 64, 4 rows 41, 38 (20, 19), 64
  // rows 64, 72 (27, 20); V = 4000 at rank 64, 4 rows 43, 36 (19, 19), 64 rows
  // 60, 39 (23, 19).  So the chain pays where W2 is long and read again; the
  // short and the single ones it takes too cost up to half as much again.
  const int cus = device_cus();
  if (p.greedy && cus > 0 && tile_path(logits_dtype, weight_dtype, V, r, base_logits, processed_logits, w1, w2) &&
      B <= dspark::chain_max_rows() && M <= kChainMaxSteps && (V + 31) / 32 <= (int64_t)cus * dspark::chain_waves_per_group() &&
      (p.r.bias == nullptr || p.r.bias_stride == 0)) {
    Control* const ctl = (Control*)workspace;
    dspark::ChainParams c{};
    c.base = base_logits;
    c.out = processed_logits;
    c.first_prev = first_prev_token_ids;
    c.tokens = sampled_tokens;
    c.w1 = (const uint16_t*)w1;
    c.w2 = (const uint16_t*)w2;
    c.sync = (uint32_t*)((char*)workspace + kControlBytes);
    c.keys = (uint64_t*)((char*)c.sync + dspark::kChainSyncBytes);
    c.bad_rows = &ctl->bad_rows;
    c.sync_failures = &ctl->sync_failures;
    c.test_hook = &ctl->chain_test_hook;
    c.B = B;
    c.M = M;
    c.V = V;
    c.r = r;
    c.S = (V + 31) / 32;
    c.rules = true;
    c.rule_set = p.r;
    c.seen = p.seen;
    c.counts = counts;
    c.mask_bytes = mask_bytes;
    e = dspark::launch_chain_greedy(c, cus, s);
    if (e == hipSuccess) return DSPARK_OK;
    (void)hipGetLastError();  // not launchable here: a launch per position
  }
  if (!table) {
    e = dspark::launch_fill_zero(keys, (size_t)B * dspark::kStepGroups * sizeof(uint64_t), s);
    if (e != hipSuccess) return device_failure(e, "step keys clear");
  }
  for (int64_t k = 0; k < M; ++k) {
    p.k = k;
    p.k_abs = (uint32_t)(position_offset + k);
    e = dspark::launch_rule_step(p, logits_dtype == DSPARK_BF16, weight_dtype == DSPARK_BF16, cus > 0 ? cus : 1, s);
    if (e != hipSuccess) return device_failure(e, "rule step launch");
  }
  e = dspark::launch_rule_choose(keys, B, M, sampled_tokens, s);
  if (e != hipSuccess) return device_failure(e, "token choice launch");
  return DSPARK_OK;
}

}  // extern "C"
