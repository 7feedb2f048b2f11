/* Sanitizer driver for the host side of the 8-bit head and the logit rules
 * (test infrastructure).  Built host-only with -fsanitize=address,undefined by
 * tests/test_sanitizers_serving.py: workspace sizes, and calls that the host
 * validation must reject, with sizes and strides at the ends of their types,
 * so that no call reaches a kernel launch: it runs without a GPU.  Exit 0
 * when every status is the expected one. */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "dspark_markov.h"

static int failures = 0;
static char fake[4096] __attribute__((aligned(256)));   /* never dereferenced: every call is rejected */
#define F ((void*)fake)
#define FI ((int64_t*)fake)
#define FF ((float*)fake)
#define AT(n) ((void*)((uintptr_t)(n) << 32))           /* addresses 4 GiB apart */

static void expect(const char* what, dspark_status_t got, dspark_status_t want) {
  if (got != want) {
    fprintf(stderr, "%s: %s, expected %s (%s)\n", what, dspark_status_string(got), dspark_status_string(want),
            dspark_markov_last_error());
    ++failures;
  }
}

static void expect_size(const char* what, size_t got, size_t want) {
  if (got != want) {
    fprintf(stderr, "%s: %zu bytes, expected %zu\n", what, got, want);
    ++failures;
  }
}

static const dspark_dtype_t bf = DSPARK_BF16, f32 = DSPARK_F32;
static const int64_t sizes[] = {INT64_MIN, INT64_MIN + 1, -(1ll << 62), -(1ll << 32), -1, 0, 1, 2, 31, 32, 33, 1ll << 16,
                                (1ll << 24) - 1, 1ll << 24, 1ll << 30, (1ll << 31) - 1, 1ll << 31, 1ll << 32, 1ll << 40, 1ll << 60,
                                1ll << 61, 1ll << 62, INT64_MAX - 1, INT64_MAX};
#define NS ((int)(sizeof(sizes) / sizeof(sizes[0])))

static dspark_status_t process(const dspark_logit_rules_t* r, int64_t B, int64_t M, int64_t V, void* out) {
  return dspark_markov_process_block(AT(1), f32, NULL, r, B, M, V, out, NULL);
}

int main(void) {
  dspark_logit_rules_t none, r;
  memset(&none, 0, sizeof none);

  /* workspace sizes: every pair of extreme sizes is answered, never wrapped */
  for (int i = 0; i < NS; ++i)
    for (int j = 0; j < NS; ++j) {
      const size_t a = dspark_markov_lm_head_int8_workspace_bytes(sizes[i], sizes[j], 5120);
      const size_t b = dspark_markov_processed_workspace_bytes(sizes[i], 4, sizes[j], 64);
      const size_t c = dspark_markov_processed_workspace_bytes(sizes[i], sizes[j], 1000, 64);
      if (a == 0 || b == 0 || c == 0) ++failures;
      if (sizes[i] > 0 && sizes[j] > 0 && sizes[i] > (INT64_MAX >> 13) / sizes[j])
        expect_size("8-bit head, sizes past the address space", a, SIZE_MAX);
    }
  expect_size("drafts, sizes past the address space", dspark_markov_processed_workspace_bytes(1ll << 40, 1, 1ll << 30, 8), SIZE_MAX);
  expect_size("a hidden size past the sums", dspark_markov_lm_head_int8_workspace_bytes(4, 4, 131073),
              dspark_markov_lm_head_int8_workspace_bytes(0, 4, INT64_MIN));

  /* sizes: with no output to write, whatever is not refused before is refused there */
  for (int i = 0; i < NS; ++i)
    for (int j = 0; j < NS; ++j) {
      const int64_t x = sizes[i], y = sizes[j];
      dspark_status_t s = dspark_markov_quantize_rows(F, bf, x, y, NULL, NULL, NULL);
      if (s == DSPARK_OK && x != 0) ++failures;
      s = dspark_markov_lm_head_int8(F, bf, 64, (int8_t*)F, FF, x, y, 1000, NULL, f32, F, SIZE_MAX, NULL);
      if (s == DSPARK_OK && x != 0 && y != 0) ++failures;
      s = dspark_markov_lm_head_int8(F, bf, x, (int8_t*)F, FF, 2, 2, y, NULL, f32, F, SIZE_MAX, NULL);
      if (s == DSPARK_OK && y != 0) ++failures;
      s = process(&none, x, y, 1000, NULL);
      if (s == DSPARK_OK && x != 0 && y != 0) ++failures;
      s = process(&none, 2, x, y, NULL);
      if (s == DSPARK_OK && x != 0 && y != 0) ++failures;
      s = dspark_markov_process_block_backward(F, F, bf, NULL, &none, x, y, 1000, NULL, NULL);
      if (s == DSPARK_OK && x != 0 && y != 0) ++failures;
      s = dspark_markov_sample_block_processed(F, bf, FI, F, F, bf, &none, x, 2, y, 64, 0.0, 0, 0, 0, NULL, F, F, SIZE_MAX, NULL);
      if (s == DSPARK_OK && x != 0) ++failures;
      s = dspark_markov_sample_block_processed(F, bf, FI, F, F, bf, &none, 2, x, 1000, y, 0.0, 0, 0, 0, NULL, F, F, SIZE_MAX, NULL);
      if (s == DSPARK_OK && x != 0) ++failures;
    }

  /* strides and lengths: extents that cannot be represented, or that reach the output */
  for (int i = 0; i < NS; ++i)
    for (int j = 0; j < NS; ++j) {
      const int64_t x = sizes[i], y = sizes[j];
      r = none;
      r.history = (const int64_t*)AT(8);
      r.history_len = x;
      r.history_stride = y;
      if (process(&r, 3, 2, 1000, NULL) != DSPARK_ERR_INVALID_ARGUMENT) ++failures;
      if (x > 0 && y >= x && y > (INT64_MAX >> 4)) expect("history past the address space", process(&r, 3, 2, 1000, AT(2)),
                                                          DSPARK_ERR_INVALID_ARGUMENT);
      r = none;
      r.logit_bias = AT(8);
      r.bias_dtype = f32;
      r.bias_stride = x;
      if (process(&r, 3, 2, 1000, NULL) != DSPARK_ERR_INVALID_ARGUMENT) ++failures;
      if (x < 0 || (x > 0 && x < 1000)) expect("bias rows over each other", process(&r, 3, 2, 1000, AT(2)), DSPARK_ERR_INVALID_ARGUMENT);
      r = none;
      r.token_mask = (const uint32_t*)AT(8);
      r.mask_stride_b = x;
      r.mask_stride_m = y;
      if (process(&r, 3, 2, 1000, NULL) != DSPARK_ERR_INVALID_ARGUMENT) ++failures;
      if (x < 0 || y < 0 || x > (INT64_MAX >> 3) || y > (INT64_MAX >> 2))
        expect("mask strides", process(&r, 3, 2, 1000, AT(2)), DSPARK_ERR_INVALID_ARGUMENT);
    }
  r = none;
  r.token_mask = (const uint32_t*)AT(8);
  r.mask_stride_b = 1ll << 30;                          /* the second request's masks begin 4 GiB on */
  expect("mask that reaches the output", process(&r, 2, 1, 1000, AT(9)), DSPARK_ERR_INVALID_ARGUMENT);
  r = none;
  r.history = (const int64_t*)AT(8);
  r.history_len = 5;
  r.history_stride = 1ll << 29;
  expect("history that reaches the output", process(&r, 2, 1, 1000, AT(9)), DSPARK_ERR_INVALID_ARGUMENT);
  r = none;
  r.logit_bias = AT(8);
  r.bias_dtype = bf;
  r.bias_stride = 1ll << 31;
  expect("biases that reach the output", process(&r, 2, 1, 1000, AT(9)), DSPARK_ERR_INVALID_ARGUMENT);

  /* the rest of the refusals */
  expect("process no rules", process(NULL, 2, 2, 10, AT(2)), DSPARK_ERR_INVALID_ARGUMENT);
  expect("backward no rules", dspark_markov_process_block_backward(F, F, bf, NULL, NULL, 2, 2, 10, AT(2), NULL),
         DSPARK_ERR_INVALID_ARGUMENT);
  expect("sample no rules", dspark_markov_sample_block_processed(F, bf, FI, F, F, bf, NULL, 2, 2, 64, 8, 0.0, 0, 0, 0, FI, F, F,
                                                                 SIZE_MAX, NULL), DSPARK_ERR_INVALID_ARGUMENT);
  expect("sample NaN temperature", dspark_markov_sample_block_processed(F, bf, FI, F, F, bf, &none, 2, 2, 64, 8, NAN, 0, 0, 0, FI,
                                                                        F, F, SIZE_MAX, NULL), DSPARK_ERR_INVALID_ARGUMENT);
  expect("sample small workspace", dspark_markov_sample_block_processed(F, bf, FI, F, F, bf, &none, 2, 2, 64, 8, 0.0, 0, 0, 0, FI,
                                                                        F, F, 8, NULL), DSPARK_ERR_WORKSPACE_TOO_SMALL);
  expect("8-bit head small workspace", dspark_markov_lm_head_int8(F, bf, 64, (int8_t*)F, FF, 2, 2, 100, F, f32, F, 8, NULL),
         DSPARK_ERR_WORKSPACE_TOO_SMALL);

  if (failures) {
    fprintf(stderr, "%d unexpected statuses\n", failures);
    return 1;
  }
  printf("serving driver: all statuses as expected\n");
  return 0;
}
