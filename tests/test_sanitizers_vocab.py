"""The host code of the 4-bit head, of sampling under limits and of the
distillation loss under AddressSanitizer and UndefinedBehaviorSanitizer (CPU
only): tests/sanitize/vocab_driver.c with their translation unit rebuilt
host-only and linked against the built library for the launchers it would
call."""
import os
import subprocess

import pytest

from tests.test_sanitizers import ENV, ROCM, ROOT, SAN, _check_clean, _run


def test_vocab_host_code_under_sanitizers(tmp_path):
    hipcc = os.path.join(ROCM, "bin", "hipcc")
    clang = os.path.join(ROCM, "llvm", "bin", "clang")
    lib_dir = os.path.join(ROOT, "rank_markov_draft_amd")
    if not (os.path.exists(hipcc) and os.path.exists(clang)):
        pytest.skip("ROCm compilers not available")
    if not os.path.exists(os.path.join(lib_dir, "libdspark_markov.so")):
        pytest.skip("libdspark_markov.so is not built")
    units, csrc = [], os.path.join(lib_dir, "csrc")
    for name in ("dspark_vocab", "dspark_markov"):   # the second holds what both share
        units.append(str(tmp_path / (name + ".o")))
        _run([hipcc, "--offload-arch=gfx950", "--cuda-host-only", "-O1", "-g", "-std=c++17", "-ffp-contract=off",
              "-I", os.path.join(ROOT, "include"), "-Xarch_host", "-fsanitize=address", "-Xarch_host",
              "-fsanitize=undefined", "-fno-omit-frame-pointer", "-c", os.path.join(csrc, name + ".hip"), "-o", units[-1]])
    drv, exe = str(tmp_path / "vocab_driver.o"), str(tmp_path / "vocab_driver")
    _run([clang, "-O1", "-g", "-fsanitize=address,undefined", "-fno-omit-frame-pointer", "-I",
          os.path.join(ROOT, "include"), "-c", os.path.join(SAN, "vocab_driver.c"), "-o", drv])
    _run([clang + "++", "-fsanitize=address,undefined", drv, *units, "-L" + lib_dir, "-ldspark_markov",
          "-Wl,-rpath," + lib_dir, "-L" + os.path.join(ROCM, "lib"), "-lamdhip64",
          "-Wl,-rpath," + os.path.join(ROCM, "lib"), "-o", exe])
    p = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=ENV)
    assert p.returncode == 0, p.stdout + p.stderr
    assert "all statuses as expected" in p.stdout
    _check_clean(p)
