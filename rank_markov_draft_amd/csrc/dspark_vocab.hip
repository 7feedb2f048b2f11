// dspark_vocab.hip -- host side of the 4-bit vocabulary head, of sampling under
// a request's limits and of the distillation loss (include/dspark_markov.h):
// argument validation, workspace layout and launches.
#include <hip/hip_runtime.h>

#include <cmath>

#include "distill.h"
#include "dspark_markov.h"
#include "fp4_head.h"
#include "host_common.h"
#include "markov_kernels.h"
#include "token_filter.h"

namespace {

using namespace dspark::host;

// Rows of codes and scales that a call makes of its hidden states: whole
// chunks of the product.
int64_t fp4_row_bytes(int64_t d) { return round_up(16 * dspark::fp4_blocks(d), dspark::kFp4K); }
size_t fp4_codes_bytes(int64_t rows, int64_t d) { return align256(mul_sz((size_t)rows, (size_t)fp4_row_bytes(d))); }
size_t fp4_scales_bytes(int64_t rows, int64_t d) { return align256(mul_sz((size_t)rows, (size_t)fp4_row_bytes(d) / 16)); }

// Checks that quantising and its inverse share; *blocks: of all rows.
dspark_status_t check_fp4(dspark_dtype_t dtype, int64_t rows, int64_t d, int64_t* blocks) {
  if (!known_dtype(dtype) || rows < 0 || d < 0) return DSPARK_ERR_INVALID_ARGUMENT;
  if (d > dspark::kFp4MaxInner) {
    dspark::set_last_error("4-bit blocks: rows must have at most 1048576 numbers");
    return DSPARK_ERR_UNSUPPORTED;
  }
  int64_t t = 0;
  if (!mul_ok(rows, dspark::fp4_blocks(d), blocks) || !mul_ok(*blocks, 128, &t)) return DSPARK_ERR_INVALID_ARGUMENT;
  return DSPARK_OK;
}
bool fp4_aligned(const void* codes, const void* scales) { return aligned16(codes) && ((uintptr_t)scales & 3u) == 0; }

// Whether a call's scratch, the workspace from kDataOffset to its `need` bytes,
// can be used: aligned, and apart from what the call reads (and writes).
bool scratch_ok(const void* workspace, size_t need, const Ranges& others) {
  return aligned16(workspace) && !others.meet((const char*)workspace + kDataOffset, need - kDataOffset);
}

// What both passes of the distillation loss check; nothing to do: *empty.
dspark_status_t check_distill(const void* logits, dspark_dtype_t dtype, const int64_t* ids, const void* teacher,
                              dspark_dtype_t teacher_dtype, int64_t B, int64_t M, int64_t V, int64_t K, double tau,
                              dspark::DistillParams* p, Ranges* in, size_t* lbytes, bool* empty) {
  if (!known_dtype(dtype) || !known_dtype(teacher_dtype) || B < 0 || M < 0 || V < 0 || K < 0)
    return DSPARK_ERR_INVALID_ARGUMENT;
  int64_t rows = 0, elems = 0, t = 0;
  if (!mul_ok(B, M, &rows) || !mul_ok(rows, V, &elems) || !mul_ok(elems, 4, &t) || !mul_ok(rows, K, &t) ||
      !mul_ok(t, 8, &t) || !mul_ok(rows, 16, &t))
    return DSPARK_ERR_INVALID_ARGUMENT;
  // the kernels hold log2(e) / tau in fp32
  const float kappa = (float)(1.4426950408889634 / tau);
  if (!(tau > 0.0) || !std::isnormal(kappa)) return DSPARK_ERR_INVALID_ARGUMENT;
  if (V > ((int64_t)1 << 30) || K > dspark::kDistillMaxEntries) return DSPARK_ERR_UNSUPPORTED;
  *empty = rows == 0;
  if (*empty) return DSPARK_OK;
  if (V == 0 || !logits || (K > 0 && (!ids || !teacher))) return DSPARK_ERR_INVALID_ARGUMENT;
  *lbytes = (size_t)elems * dtype_bytes(dtype);
  in->add(ids, (size_t)(rows * K) * sizeof(int64_t));
  in->add(teacher, (size_t)(rows * K) * dtype_bytes(teacher_dtype));
  p->logits = logits;
  p->teacher_ids = ids;
  p->teacher_logits = teacher;
  p->rows = rows;
  p->V = V;
  p->K = K;
  p->tau = tau;
  p->kappa = kappa;
  p->teacher_bf16 = teacher_dtype == DSPARK_BF16;
  return DSPARK_OK;
}

}  // namespace

extern "C" {

dspark_status_t dspark_markov_quantize_fp4(const void* x, dspark_dtype_t dtype, int64_t rows, int64_t d, uint8_t* codes,
                                           uint8_t* scales, void* stream) {
  int64_t blocks = 0;
  const dspark_status_t st = check_fp4(dtype, rows, d, &blocks);
  if (st != DSPARK_OK || blocks == 0) return st;
  if (!x || !codes || !scales || !fp4_aligned(codes, scales)) return DSPARK_ERR_INVALID_ARGUMENT;
  const size_t xb = (size_t)(rows * d) * dtype_bytes(dtype), cb = (size_t)blocks * 16, sb = (size_t)blocks;
  if (overlaps(codes, cb, x, xb) || overlaps(scales, sb, x, xb) || overlaps(codes, cb, scales, sb))
    return DSPARK_ERR_INVALID_ARGUMENT;
  const dspark::Fp4QuantizeParams p{x, codes, scales, rows, d, 16 * dspark::fp4_blocks(d)};
  const hipError_t e = dspark::launch_fp4_quantize(p, dtype == DSPARK_BF16, (hipStream_t)stream);
  if (e != hipSuccess) return device_failure(e, "4-bit quantize launch");
  return DSPARK_OK;
}

dspark_status_t dspark_markov_dequantize_fp4(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t d,
                                             void* x, dspark_dtype_t dtype, void* stream) {
  int64_t blocks = 0;
  const dspark_status_t st = check_fp4(dtype, rows, d, &blocks);
  if (st != DSPARK_OK || blocks == 0) return st;
  if (!x || !codes || !scales || !fp4_aligned(codes, scales)) return DSPARK_ERR_INVALID_ARGUMENT;
  const size_t xb = (size_t)(rows * d) * dtype_bytes(dtype);
  if (overlaps(codes, (size_t)blocks * 16, x, xb) || overlaps(scales, (size_t)blocks, x, xb))
    return DSPARK_ERR_INVALID_ARGUMENT;
  const dspark::Fp4DequantizeParams p{codes, scales, x, rows, d, dspark::fp4_blocks(d)};
  const hipError_t e = dspark::launch_fp4_dequantize(p, dtype == DSPARK_BF16, (hipStream_t)stream);
  if (e != hipSuccess) return device_failure(e, "4-bit dequantize launch");
  return DSPARK_OK;
}

size_t dspark_markov_lm_head_fp4_workspace_bytes(int64_t B, int64_t M, int64_t d) {
  if (B < 0 || M < 0 || d < 0 || d > dspark::kFp4MaxInner) return kDataOffset;
  int64_t rows = 0;
  if (!mul_ok(B, M, &rows)) return SIZE_MAX;
  return add_sz(kDataOffset, add_sz(fp4_codes_bytes(rows, d), fp4_scales_bytes(rows, d)));
}

dspark_status_t dspark_markov_lm_head_fp4(const void* hidden_states, dspark_dtype_t hidden_dtype, int64_t d,
                                          const uint8_t* head_codes, const uint8_t* head_scales, int64_t B, int64_t M,
                                          int64_t V, void* logits, dspark_dtype_t logits_dtype, void* workspace,
                                          size_t workspace_bytes, void* stream) {
  if (!known_dtype(hidden_dtype) || !known_dtype(logits_dtype)) return DSPARK_ERR_INVALID_ARGUMENT;
  if (B < 0 || M < 0 || V < 0 || d <= 0) return DSPARK_ERR_INVALID_ARGUMENT;
  int64_t rows = 0, elems = 0, t = 0;
  if (!mul_ok(B, M, &rows) || !mul_ok(rows, V, &elems) || !mul_ok(elems, 4, &t)) return DSPARK_ERR_INVALID_ARGUMENT;
  if (d > dspark::kFp4MaxInner) {
    dspark::set_last_error("lm_head_fp4: the hidden size must be at most 1048576");
    return DSPARK_ERR_UNSUPPORTED;
  }
  if (!mul_ok(V, fp4_row_bytes(d), &t) || !mul_ok(rows, fp4_row_bytes(d), &t) || !mul_ok(rows, d, &t) || !mul_ok(t, 4, &t))
    return DSPARK_ERR_INVALID_ARGUMENT;
  if (rows > (int64_t)0x7FFFFFFF || V > (int64_t)0x7FFFFFFF) return DSPARK_ERR_UNSUPPORTED;
  if (elems == 0) return DSPARK_OK;
  if (!hidden_states || !head_codes || !head_scales || !logits || !fp4_aligned(head_codes, head_scales))
    return DSPARK_ERR_INVALID_ARGUMENT;
  const size_t need = dspark_markov_lm_head_fp4_workspace_bytes(B, M, d);
  if (!workspace || workspace_bytes < need) return DSPARK_ERR_WORKSPACE_TOO_SMALL;
  const int64_t blocks = dspark::fp4_blocks(d);
  Ranges in;
  in.add(hidden_states, (size_t)(rows * d) * dtype_bytes(hidden_dtype));
  in.add(head_codes, (size_t)(V * blocks * 16));
  in.add(head_scales, (size_t)(V * blocks));
  if (in.meet(logits, (size_t)elems * dtype_bytes(logits_dtype))) return DSPARK_ERR_INVALID_ARGUMENT;
  in.add(logits, (size_t)elems * dtype_bytes(logits_dtype));
  if (!scratch_ok(workspace, need, in)) return DSPARK_ERR_INVALID_ARGUMENT;
  const hipStream_t s = (hipStream_t)stream;
  uint8_t* const xc = (uint8_t*)workspace + kDataOffset;
  uint8_t* const xs = xc + fp4_codes_bytes(rows, d);
  const dspark::Fp4QuantizeParams q{hidden_states, xc, xs, rows, d, fp4_row_bytes(d)};
  hipError_t e = dspark::launch_fp4_quantize(q, hidden_dtype == DSPARK_BF16, s);
  if (e != hipSuccess) return device_failure(e, "hidden state quantize launch");
  const dspark::Fp4HeadParams p{xc, xs, head_codes, head_scales, logits, rows, V, blocks, fp4_row_bytes(d)};
  e = dspark::launch_fp4_head(p, logits_dtype == DSPARK_BF16, device_cus(), s);
  if (e == hipErrorNotSupported) {
    (void)hipGetLastError();
    return DSPARK_ERR_UNSUPPORTED;
  }
  if (e != hipSuccess) return device_failure(e, "fp4 head launch");
  return DSPARK_OK;
}

size_t dspark_markov_sample_filtered_workspace_bytes(int64_t B, int64_t M, int64_t V) {
  if (B < 0 || M < 0 || V < 0) return kDataOffset;
  int64_t rows = 0;
  if (!mul_ok(B, M, &rows)) return SIZE_MAX;
  const size_t groups = mul_sz((size_t)rows, (size_t)(V / dspark::kFilterGroup + 1));
  return add_sz(kDataOffset, add_sz(align256(mul_sz(groups, sizeof(double))), align256(mul_sz(groups, sizeof(uint32_t)))));
}

dspark_status_t dspark_markov_sample_filtered(const void* logits, dspark_dtype_t logits_dtype, const float* uniforms,
                                              const dspark_token_limits_t* limits, int64_t B, int64_t M, int64_t V,
                                              int64_t* tokens, float* probs, void* workspace, size_t workspace_bytes,
                                              void* stream) {
  if (!known_dtype(logits_dtype) || B < 0 || M < 0 || V < 0 || !limits) return DSPARK_ERR_INVALID_ARGUMENT;
  int64_t rows = 0, elems = 0, t = 0;
  if (!mul_ok(B, M, &rows) || !mul_ok(rows, V, &elems) || !mul_ok(elems, 4, &t) || !mul_ok(rows, 8, &t))
    return DSPARK_ERR_INVALID_ARGUMENT;
  if (V > ((int64_t)1 << 30)) return DSPARK_ERR_UNSUPPORTED;
  if (rows == 0) return DSPARK_OK;
  if (V == 0 || !logits || !uniforms || !tokens || !probs) return DSPARK_ERR_INVALID_ARGUMENT;
  const size_t need = dspark_markov_sample_filtered_workspace_bytes(B, M, V);
  if (!workspace || workspace_bytes < need) return DSPARK_ERR_WORKSPACE_TOO_SMALL;
  const size_t tb = (size_t)rows * sizeof(int64_t), pb = (size_t)rows * sizeof(float), vb = (size_t)B * sizeof(float);
  Ranges in;
  in.add(logits, (size_t)elems * dtype_bytes(logits_dtype));
  in.add(uniforms, pb);
  in.add(limits->temperature, vb);
  in.add(limits->top_k, (size_t)B * sizeof(int64_t));
  in.add(limits->top_p, vb);
  in.add(limits->min_p, vb);
  if (in.meet(tokens, tb) || in.meet(probs, pb) || overlaps(tokens, tb, probs, pb)) return DSPARK_ERR_INVALID_ARGUMENT;
  in.add(tokens, tb);
  in.add(probs, pb);
  if (!scratch_ok(workspace, need, in)) return DSPARK_ERR_INVALID_ARGUMENT;
  dspark::FilterParams p{};
  p.limits = dspark::TokenLimits{limits->temperature,   limits->top_k,           limits->top_p,     limits->min_p,
                                 limits->all_top_k,     limits->all_temperature, limits->all_top_p, limits->all_min_p};
  p.logits = logits;
  p.uniforms = uniforms;
  p.tokens = tokens;
  p.probs = probs;
  p.sums = (double*)((char*)workspace + kDataOffset);
  p.tops = (uint32_t*)((char*)p.sums + align256((size_t)rows * (size_t)(V / dspark::kFilterGroup + 1) * sizeof(double)));
  p.rows = rows;
  p.M = M;
  p.V = V;
  const hipError_t e = dspark::launch_token_filter(p, logits_dtype == DSPARK_BF16, (hipStream_t)stream);
  if (e != hipSuccess) return device_failure(e, "filtered sampling launch");
  return DSPARK_OK;
}

size_t dspark_markov_distill_workspace_bytes(int64_t B, int64_t M, int64_t V) {
  if (B < 0 || M < 0 || V < 0) return kDataOffset;
  int64_t rows = 0;
  if (!mul_ok(B, M, &rows)) return SIZE_MAX;
  // a slice's two numbers: rows * distill_slices(rows, V) of them at most, in a
  // form that no smaller call exceeds
  const size_t all = mul_sz((size_t)rows, (size_t)dspark::distill_slices(1, V)), some = add_sz((size_t)rows, 2048);
  return add_sz(kDataOffset, align256(mul_sz(all < some ? all : some, 2 * sizeof(float))));
}

dspark_status_t dspark_markov_distill_block(const void* logits, dspark_dtype_t logits_dtype, const int64_t* teacher_ids,
                                            const void* teacher_logits, dspark_dtype_t teacher_dtype, int64_t B,
                                            int64_t M, int64_t V, int64_t K, double temperature, float* loss,
                                            float* stats, void* workspace, size_t workspace_bytes, void* stream) {
  dspark::DistillParams p{};
  Ranges in;
  size_t lbytes = 0;
  bool empty = false;
  const dspark_status_t st = check_distill(logits, logits_dtype, teacher_ids, teacher_logits, teacher_dtype, B, M, V, K,
                                           temperature, &p, &in, &lbytes, &empty);
  if (st != DSPARK_OK || empty) return st;
  if (!loss || !stats) return DSPARK_ERR_INVALID_ARGUMENT;
  const size_t need = dspark_markov_distill_workspace_bytes(B, M, V);
  if (!workspace || workspace_bytes < need) return DSPARK_ERR_WORKSPACE_TOO_SMALL;
  const size_t rb = (size_t)p.rows * sizeof(float);
  in.add(logits, lbytes);
  if (in.meet(loss, rb) || in.meet(stats, 4 * rb) || overlaps(loss, rb, stats, 4 * rb)) return DSPARK_ERR_INVALID_ARGUMENT;
  in.add(loss, rb);
  in.add(stats, 4 * rb);
  if (!scratch_ok(workspace, need, in)) return DSPARK_ERR_INVALID_ARGUMENT;
  p.loss = loss;
  p.stats = stats;
  p.partials = (float*)((char*)workspace + kDataOffset);
  const hipError_t e = dspark::launch_distill_loss(p, logits_dtype == DSPARK_BF16, (hipStream_t)stream);
  if (e != hipSuccess) return device_failure(e, "distillation loss launch");
  return DSPARK_OK;
}

dspark_status_t dspark_markov_distill_block_backward(const float* grad_loss, const void* logits,
                                                     dspark_dtype_t logits_dtype, const int64_t* teacher_ids,
                                                     const void* teacher_logits, dspark_dtype_t teacher_dtype,
                                                     const float* stats, int64_t B, int64_t M, int64_t V, int64_t K,
                                                     double temperature, void* grad_logits, void* stream) {
  dspark::DistillParams p{};
  Ranges in;
  size_t lbytes = 0;
  bool empty = false;
  const dspark_status_t st = check_distill(logits, logits_dtype, teacher_ids, teacher_logits, teacher_dtype, B, M, V, K,
                                           temperature, &p, &in, &lbytes, &empty);
  if (st != DSPARK_OK || empty) return st;
  if (!grad_loss || !stats || !grad_logits) return DSPARK_ERR_INVALID_ARGUMENT;
  const size_t rb = (size_t)p.rows * sizeof(float);
  in.add(grad_loss, rb);
  in.add(stats, 4 * rb);
  if (in.meet(grad_logits, lbytes)) return DSPARK_ERR_INVALID_ARGUMENT;
  if (grad_logits != logits && overlaps(grad_logits, lbytes, logits, lbytes)) return DSPARK_ERR_INVALID_ARGUMENT;
  p.grad_loss = grad_loss;
  p.stats = const_cast<float*>(stats);
  p.grad = grad_logits;
  const hipError_t e = dspark::launch_distill_backward(p, logits_dtype == DSPARK_BF16, (hipStream_t)stream);
  if (e != hipSuccess) return device_failure(e, "distillation gradient launch");
  return DSPARK_OK;
}

}  // extern "C"
