// dspark_vocab.hip -- host side of the 4-bit vocabulary head
// (include/dspark_markov.h): argument validation, workspace layout and
// launches.
#include <hip/hip_runtime.h>

#include "dspark_markov.h"
#include "fp4_head.h"
#include "host_common.h"
#include "markov_kernels.h"

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
  if (!workspace || workspace_bytes < dspark_markov_lm_head_fp4_workspace_bytes(B, M, d))
    return DSPARK_ERR_WORKSPACE_TOO_SMALL;
  const int64_t blocks = dspark::fp4_blocks(d);
  Ranges in;
  in.add(hidden_states, (size_t)(rows * d) * dtype_bytes(hidden_dtype));
  in.add(head_codes, (size_t)(V * blocks * 16));
  in.add(head_scales, (size_t)(V * blocks));
  if (in.meet(logits, (size_t)elems * dtype_bytes(logits_dtype))) return DSPARK_ERR_INVALID_ARGUMENT;
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

}  // extern "C"
