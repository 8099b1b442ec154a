"""CPU test of the built library's code: the 16-bit products' matrix instructions are
written as inline assembly, around which the compiler adds none of the wait
states that gfx950 needs between vector and matrix instructions.  Disassembled,
in every tiled kernel of theirs
  - a vector instruction that writes an operand of a matrix instruction comes two
    wait states before it at least;
  - an instruction other than a matrix one that reads or writes a matrix
    instruction's result comes eleven wait states (16 x 16 x 32) after it at least;
  - a fragment that an LDS read brings has been waited for."""
import os
import re
import shutil
import subprocess

import pytest

import fp4_gemm_moe_amd as hq
from fp4_gemm_moe_amd import build

BEFORE, AFTER = 2, 11


def _regs(operand):
    """The vector registers ('v' or 'a', number) that an operand names."""
    m = re.fullmatch(r"([va])\[(\d+):(\d+)\]", operand)
    if m:
        return {(m[1], i) for i in range(int(m[2]), int(m[3]) + 1)}
    m = re.fullmatch(r"([va])(\d+)", operand)
    return {(m[1], int(m[2]))} if m else set()


def _violations(listing):
    """(matrix instructions, descriptions of what comes too early) of a listing."""
    count, bad = 0, []
    history = []            # (text, wait states, vector registers written by vector code, results of a matrix instruction)
    pending = []            # registers of LDS reads under way, oldest first
    for line in listing:
        text = line.split("//")[0].strip()
        if not text or text.endswith(":"):
            continue
        op, _, rest = text.partition(" ")
        operands = [o for part in rest.split(",") for o in part.split()]
        regs = [_regs(o) for o in operands]
        every = set().union(*regs) if regs else set()
        matrix = op.startswith("v_mfma")
        if op == "s_waitcnt":
            m = re.search(r"lgkmcnt\((\d+)\)", rest)
            if m:
                pending = pending[len(pending) - int(m[1]):] if int(m[1]) < len(pending) else pending
                pending = [] if int(m[1]) == 0 else pending
        if matrix:
            count += 1
            if every & set().union(*pending):
                bad.append(f"{text}: an LDS read has not been waited for")
        states = 0
        for prev, length, written, result in reversed(history):
            if matrix and states < BEFORE and written & every:
                bad.append(f"{prev} -> {text} ({states} wait states)")
            if not matrix and states < AFTER and result & every:
                bad.append(f"{prev} -> {text} ({states} wait states)")
            states += length
            if states >= AFTER:
                break
        if op.startswith("ds_"):
            reads = "read" in op
            pending.append(regs[0] if reads and regs else set())
        elif op.startswith("s_load") or op.startswith("s_buffer_load"):
            pending.append(set())
        length = int(operands[0]) + 1 if op == "s_nop" else 1
        written = regs[0] if op.startswith("v_") and not matrix and regs else set()
        history = history[-24:] + [(text, length, written, regs[0] if matrix else set())]
    return count, bad


def test_the_rules_on_short_listings():
    mul = "v_mfma_f32_16x16x32_bf16 a[0:3], v[0:3], v[4:7], a[0:3]"
    assert _violations(["v_mov_b32 v1, 0", "s_nop 0", mul])[1]
    assert _violations(["v_accvgpr_write_b32 a2, v9", "s_nop 1", mul]) == (1, [])
    assert _violations([mul, "s_nop 9", "v_accvgpr_read_b32 v9, a3"])[1]
    assert _violations([mul, "s_nop 10", "v_accvgpr_read_b32 v9, a3"]) == (1, [])
    assert _violations([mul, mul]) == (2, [])
    read = "ds_read_b128 v[4:7], v9"
    assert _violations([read, mul])[1]
    assert _violations([read, "ds_read_b128 v[20:23], v9", "s_waitcnt lgkmcnt(1)", mul]) == (1, [])
    assert _violations(["ds_read_b128 v[20:23], v9", read, "s_waitcnt lgkmcnt(1)", mul])[1]


def test_products_wait(tmp_path):
    tool = shutil.which("llvm-objdump") or os.path.join(os.path.dirname(os.path.dirname(build.HIPCC)),
                                                        "llvm", "bin", "llvm-objdump")
    if not os.path.exists(tool):
        pytest.skip("no disassembler")
    if not os.path.exists(hq.library_path()):
        build.build(verbose=False)
    shutil.copy(hq.library_path(), tmp_path / "lib.so")
    subprocess.run([tool, "--offloading", "lib.so"], cwd=tmp_path, check=True, capture_output=True)
    count, bad = 0, []
    for f in sorted(tmp_path.glob("lib.so.*gfx950")):
        out = subprocess.run([tool, "-d", "--no-show-raw-insn", str(f)], check=True, capture_output=True, text=True).stdout
        for part in re.split(r"\n(?=[0-9a-f]+ <[^>]*>:\n)", out):
            if "half_gemm_tiled" not in part.split("\n", 1)[0]:
                continue
            n, b = _violations(part.splitlines()[1:])
            count += n
            bad += b
    assert count > 0
    assert not bad, f"{len(bad)} of {count} matrix instructions, first: {bad[:3]}"
