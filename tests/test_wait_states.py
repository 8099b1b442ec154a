"""CPU test of the built library's code: the loads from memory into LDS are
written as inline assembly, inside and before which the compiler adds none of the
wait states that gfx9 hardware needs.  Disassembled, each of them has
  - one wait state at least between the scalar write of m0, its LDS address,
    and the load;
  - five at least between a vector instruction's write of a scalar register
    and the load, if that reads it."""
import os
import re
import shutil
import subprocess

import pytest

import fp4_gemm_moe_amd as hq
from fp4_gemm_moe_amd import build

M0_STATES, SGPR_STATES = 1, 5


def _scalars(operand):
    """The numbers of the scalar registers that an operand names."""
    m = re.fullmatch(r"s\[(\d+):(\d+)\]", operand)
    if m:
        return set(range(int(m[1]), int(m[2]) + 1))
    m = re.fullmatch(r"s(\d+)", operand)
    return {int(m[1])} if m else set()


def _violations(listing):
    """(loads into LDS, descriptions of those that come too early) of a listing."""
    loads, bad, history = 0, [], []           # history: (text, wait states, writes m0, scalars written by vector code)
    for line in listing:
        text = line.split("//")[0].strip()
        if not text or text.endswith(":"):
            continue
        op, _, rest = text.partition(" ")
        operands = [o for part in rest.split(",") for o in part.split()]
        if op.startswith("buffer_load") and operands[-1] == "lds":
            loads += 1
            read, states = set().union(*map(_scalars, operands)), 0
            for prev, length, sets_m0, written in reversed(history):
                if states < M0_STATES and sets_m0 or states < SGPR_STATES and written & read:
                    bad.append(f"{prev} -> {text} ({states} wait states)")
                states += length
                if states >= SGPR_STATES:
                    break
        vector = set()
        if op.startswith("v_") and operands:
            vector = _scalars(operands[0])
            if "_co_" in op or op.startswith("v_div_scale"):
                vector |= _scalars(operands[1])
        length = int(operands[0]) + 1 if op == "s_nop" else 1
        history = history[-7:] + [(text, length, op.startswith("s_") and bool(operands) and operands[0] == "m0", vector)]
    return loads, bad


def test_the_rules_on_short_listings():
    load = "buffer_load_dwordx4 v1, s[4:7], s3 offen lds // 0001"
    assert _violations(["s_mov_b32 m0, s2", load])[1]
    assert _violations(["s_mov_b32 m0, s2", "s_nop 0", load]) == (1, [])
    assert _violations(["s_mov_b32 m0, s2", "s_mov_b32 s9, s8", load]) == (1, [])
    first = "v_readfirstlane_b32 s6, v2"
    assert _violations([first, "s_nop 3", load])[1]
    assert _violations([first, "s_nop 4", load]) == (1, [])
    assert _violations(["v_readfirstlane_b32 s8, v2", load]) == (1, [])
    assert _violations(["v_cmp_lt_u32_e64 s[2:3], v1, v2", "s_nop 0", load])[1]
    assert _violations(["buffer_load_dwordx4 v1, s[4:7], s3 offen"]) == (0, [])


def test_loads_into_lds_wait(tmp_path):
    tool = shutil.which("llvm-objdump") or os.path.join(os.path.dirname(os.path.dirname(build.HIPCC)),
                                                        "llvm", "bin", "llvm-objdump")
    if not os.path.exists(tool):
        pytest.skip("no disassembler")
    if not os.path.exists(hq.library_path()):
        build.build(verbose=False)
    shutil.copy(hq.library_path(), tmp_path / "lib.so")
    subprocess.run([tool, "--offloading", "lib.so"], cwd=tmp_path, check=True, capture_output=True)
    loads, bad = 0, []
    for f in sorted(tmp_path.glob("lib.so.*gfx950")):
        out = subprocess.run([tool, "-d", "--no-show-raw-insn", str(f)], check=True, capture_output=True, text=True)
        n, b = _violations(out.stdout.splitlines())
        loads += n
        bad += b
    assert loads > 0
    assert not bad, f"{len(bad)} of {loads} loads, first: {bad[:3]}"
