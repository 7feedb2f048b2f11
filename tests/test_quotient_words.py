"""The claim behind the greedy chain's quotients (csrc/logit_rules_device.h),
over all pairs of significands: y * high + y * low, with high and low the two
words of a penalty's reciprocal, is the division's own rounding of a bf16 value
y over the penalty, but for the two penalties that are left out (CPU only)."""
import os
import re
import shutil
import subprocess

import pytest

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "rank_markov_draft_amd", "csrc",
                      "logit_rules_device.h")
PROGRAM = r"""
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>
static float value(uint32_t significand) {
  const uint32_t b = 0x3F800000u | significand;
  float f;
  memcpy(&f, &b, 4);
  return f;
}
int main(void) {
#pragma omp parallel for
  for (uint32_t m = 0; m < 1u << 23; ++m) {
    const float rep = value(m), high = 1.0f / rep, low = fmaf(-rep, high, 1.0f) / rep;
    int off = 0;
    for (uint32_t k = 0; k < 128; ++k) {
      const float y = value(k << 16);
      off += fmaf(y, high, y * low) != y / rep;
    }
    if (off) printf("0x%X\n", m);
  }
  return 0;
}
"""


def test_every_pair_of_significands(tmp_path):
    with open("/proc/cpuinfo") as f:
        if shutil.which("gcc") is None or " fma " not in f.read():
            pytest.skip("gcc or fused products not available")
    src, exe = tmp_path / "quotients.c", str(tmp_path / "quotients")
    src.write_text(PROGRAM)
    subprocess.run(["gcc", "-O3", "-march=native", "-ffp-contract=off", "-fopenmp", str(src), "-lm", "-o", exe], check=True)
    off = set(subprocess.run([exe], check=True, capture_output=True, text=True, timeout=300).stdout.split())
    with open(HEADER) as f:
        left_out = set(re.findall(r"s == (0x[0-9A-F]+)u", f.read()))
    assert off == left_out and len(off) == 2
