"""The wait states that inline assembly has to leave by itself, counted in the
built library's gfx950 code (CPU only).

The compiler inserts the wait states its own instructions need, and does not
look into an assembly string.  The loads to LDS and the rounding conversion of
device_common.h are such strings."""
import os
import re
import shutil
import subprocess

import pytest

from rank_markov_draft_amd import _lib

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
# wait states between an instruction that writes M0 and a load to LDS, which reads it
M0_STATES = 1
# and between a vector instruction that writes a scalar register (a spilled one read back from a
# lane) and a memory instruction that reads it, as the words of its buffer
SCALAR_STATES = 5
# and between a matrix instruction of 2, 8 or 16 passes and a vector instruction that reads its
# result, as the conversion in bf16_rne may
MATRIX_STATES = {"4x4": 5, "16x16": 11, "32x32": 19}


def _wait_states(ins):
    nop = re.match(r"s_nop (\d+)", ins)
    return int(nop[1]) + 1 if nop else 1


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """{kernel: its instructions in order} of every code object in the library."""
    if not os.path.exists(OBJDUMP):
        pytest.skip("llvm-objdump not available")
    if not os.path.exists(_lib.LIB_PATH):
        _lib.build()
    d = tmp_path_factory.mktemp("code")
    lib = shutil.copy(_lib.LIB_PATH, d)
    subprocess.run([OBJDUMP, "--offloading", lib], check=True, capture_output=True, cwd=d)
    found = {}
    for name in sorted(os.listdir(d)):
        if "gfx950" not in name:
            continue
        text = subprocess.run([OBJDUMP, "-d", "--mcpu=gfx950", str(d / name)], check=True, capture_output=True, text=True).stdout
        body = None
        for line in text.splitlines():
            head = re.match(r"[0-9a-f]+ <(.+)>:", line)
            if head:
                body = found.setdefault((name, head[1]), [])
            elif line.startswith("\t") and body is not None:
                body.append(line.split("//")[0].strip())
    return found


def _lds_loads(body):
    """Index and text of the loads to LDS."""
    return [(i, ins) for i, ins in enumerate(body) if ins.startswith("buffer_load") and ins.endswith(" lds")]


def _states_since(body, i, writes):
    """Wait states between instruction i and the last of the eight before it that ``writes``."""
    states = 0
    for ins in reversed(body[max(0, i - 8):i]):
        if writes(ins):
            return states
        states += _wait_states(ins)
    return None


def test_loads_to_lds_follow_the_write_of_m0(kernels):
    loads = 0
    for where, body in kernels.items():
        for i, ins in _lds_loads(body):
            states = _states_since(body, i, lambda p: re.match(r"s_\w+ m0,", p))
            assert states is None or states >= M0_STATES, f"{where[1]}: {body[i - 1]}; {ins}"
            loads += 1
    assert loads > 0


def test_loads_to_lds_follow_their_buffer_words(kernels):
    for where, body in kernels.items():
        for i, ins in _lds_loads(body):
            first, last = (int(n) for n in re.search(r"s\[(\d+):(\d+)\]", ins).groups())

            def writes(p):
                lane = re.match(r"v_read(?:first)?lane_b32 s(\d+),", p)
                return lane and first <= int(lane[1]) <= last

            states = _states_since(body, i, writes)
            assert states is None or states >= SCALAR_STATES, f"{where[1]}: {body[max(0, i - 6):i + 1]}"


def _vectors(operands):
    """Vector registers named in a text of operands."""
    found = set()
    for first, last, one in re.findall(r"\bv\[(\d+):(\d+)\]|\bv(\d+)\b", operands):
        found.update(range(int(first), int(last) + 1) if first else [int(one)])
    return found


def test_conversions_follow_the_matrix_results_they_read(kernels):
    conversions = 0
    for where, body in kernels.items():
        pending = []  # [registers, wait states since, wait states needed] in straight-line order
        for ins in body:
            name, _, operands = ins.partition(" ")
            target, _, sources = operands.partition(",")
            if name == "v_cvt_pk_bf16_f32" and sources.split(",")[0].strip() == "0":
                conversions += 1
                for regs, states, needed in pending:
                    assert states >= needed or not regs & _vectors(sources), f"{where[1]}: {ins} after {states} wait states"
            if name.startswith("v_") and not name.startswith("v_mfma"):
                for p in pending:
                    p[0] -= _vectors(target)
            pending = [[r, s + _wait_states(ins), n] for r, s, n in pending if r and s < n]
            shape = re.match(r"v_mfma_\w+?_(\d+x\d+)x", name)
            if shape:
                pending.append([_vectors(target), 0, MATRIX_STATES[shape[1]]])
            if name in ("s_branch", "s_endpgm", "s_setpc_b64"):
                pending = []
    assert conversions > 0
