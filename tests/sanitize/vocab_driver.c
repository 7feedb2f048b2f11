/* Sanitizer driver for the host side of the 4-bit head, of sampling under
 * limits and of the distillation loss (test infrastructure).  Built host-only
 * with -fsanitize=address,undefined by tests/test_sanitizers_vocab.py:
 * workspace sizes, and calls that the host validation must reject, with sizes
 * at the ends of their types, so that no call reaches a kernel launch: it runs
 * without a GPU.  Exit 0 when every status is the expected one. */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "dspark_markov.h"

static int failures = 0;
#define AT(n) ((void*)((uintptr_t)(n) << 32))           /* addresses 4 GiB apart, never dereferenced */

static const int64_t sizes[] = {INT64_MIN, INT64_MIN + 1, -(1ll << 62), -(1ll << 32), -1, 0, 1, 2, 31, 127, 128, 129,
                                1ll << 16, 1ll << 20, (1ll << 20) + 1, (1ll << 30) + 1, (1ll << 31) - 1, 1ll << 31, 1ll << 40,
                                1ll << 58, 1ll << 60, 1ll << 62, INT64_MAX - 1, INT64_MAX};
#define NS ((int)(sizeof(sizes) / sizeof(sizes[0])))

/* Whatever the sizes, a call with a workspace of one byte is refused, or is
 * empty: nothing is launched. */
static void refused_or_empty(const char* what, dspark_status_t st, int64_t a, int64_t b, int64_t c, int empty) {
  if (st == DSPARK_ERR_DEVICE || (st == DSPARK_OK && !empty)) {
    fprintf(stderr, "%s (%lld, %lld, %lld): %s\n", what, (long long)a, (long long)b, (long long)c, dspark_status_string(st));
    ++failures;
  }
}

int main(void) {
  dspark_token_limits_t lim;
  memset(&lim, 0, sizeof lim);
  lim.all_temperature = 1.0f;
  for (int i = 0; i < NS; ++i)
    for (int j = 0; j < NS; ++j) {
      if (dspark_markov_lm_head_fp4_workspace_bytes(sizes[i], sizes[j], 5120) == 0 ||
          dspark_markov_lm_head_fp4_workspace_bytes(sizes[i], 1, sizes[j]) == 0 ||
          dspark_markov_sample_filtered_workspace_bytes(sizes[i], 3, sizes[j]) == 0 ||
          dspark_markov_distill_workspace_bytes(sizes[i], 1, sizes[j]) == 0 ||
          dspark_markov_distill_workspace_bytes(sizes[i], sizes[j], 1000) == 0)
        ++failures;
      for (int k = 0; k < NS; ++k) {
        const int64_t a = sizes[i], b = sizes[j], c = sizes[k];
        const int none = a == 0 || b == 0;
        refused_or_empty("head", dspark_markov_lm_head_fp4(AT(1), DSPARK_F32, c, AT(2), AT(3), a, 1, b, AT(4), DSPARK_F32,
                                                           AT(5), 1, NULL), a, b, c, none);
        refused_or_empty("sample", dspark_markov_sample_filtered(AT(1), DSPARK_BF16, AT(2), &lim, a, b, c, AT(3), AT(4),
                                                                 AT(5), 1, NULL), a, b, c, none);
        refused_or_empty("distill", dspark_markov_distill_block(AT(1), DSPARK_F32, AT(2), AT(3), DSPARK_F32, a, b, c, 4,
                                                                1.0, AT(4), AT(5), AT(6), 1, NULL), a, b, c, none);
        refused_or_empty("distill entries", dspark_markov_distill_block(AT(1), DSPARK_F32, AT(2), AT(3), DSPARK_F32, a, 2, b,
                                                                        c, 1.0, AT(4), AT(5), AT(6), 1, NULL), a, b, c, a == 0);
        refused_or_empty("distill backward", dspark_markov_distill_block_backward(
                             AT(7), AT(1), DSPARK_F32, AT(2), AT(3), DSPARK_F32, AT(4), a, b, c, 4, NAN, AT(5), NULL),
                         a, b, c, 0);
      }
      refused_or_empty("quantize", dspark_markov_quantize_fp4(NULL, DSPARK_F32, sizes[i], sizes[j], AT(2), AT(3), NULL),
                       sizes[i], sizes[j], 0, sizes[i] == 0 || sizes[j] == 0);
      refused_or_empty("dequantize", dspark_markov_dequantize_fp4(AT(2), NULL, sizes[i], sizes[j], AT(1), DSPARK_F32, NULL),
                       sizes[i], sizes[j], 0, sizes[i] == 0 || sizes[j] == 0);
    }
  if (failures) return 1;
  printf("all statuses as expected\n");
  return 0;
}
