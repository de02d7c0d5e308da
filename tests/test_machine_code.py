"""The built library's gfx950 code, disassembled: instructions written in
inline asm keep the wait states that the compiler keeps for its own.

The assembler adds none inside an asm statement, so the two hazards that a
copy from memory into LDS (buffer_load ... lds) can meet are looked for here
in every kernel:
  a scalar write of M0, then the copy that takes its LDS address from M0:
    one instruction (s_nop counts its operand + 1) has to lie between;
  a vector instruction that writes an SGPR (v_readfirstlane and the like),
    then a memory instruction that reads it: five."""

import os
import re
import shutil
import subprocess

import pytest

from fac_whitening_gift_amd import build as fb

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"


def _registers(operand):
    """scalar registers that an operand names"""
    m = re.fullmatch(r"s(\d+)", operand)
    if m:
        return {int(m[1])}
    m = re.fullmatch(r"s\[(\d+):(\d+)\]", operand)
    if m:
        return set(range(int(m[1]), int(m[2]) + 1))
    return {operand} if operand in ("vcc", "m0") else set()


def hazards(lines):
    """-> (copies into LDS, [(kernel, instruction, missing what)]) of a disassembly"""
    copies, found = 0, []
    kernel, past = "", []   # past: (mnemonic, scalar registers written, wait states)
    for line in lines:
        m = re.match(r"[0-9a-f]+ <(.*)>:", line)
        if m:
            kernel, past = m[1], []
            continue
        text = line.split("//")[0].strip()
        if not line.startswith("\t") or not text:
            continue
        name, *rest = text.split(None, 1)
        operands = [o.strip() for o in rest[0].split(",")] if rest else []
        if name.startswith(("buffer_", "global_", "flat_", "scratch_")):
            read = {r for o in operands for word in o.split() for r in _registers(word)}
            checks = [("v_", read, 5, "VALU write of an SGPR")]
            if re.search(r"\blds\b", text) or "_load_lds_" in name:
                copies += 1
                checks.append(("s_", {"m0"}, 1, "scalar write of M0"))
            for kind, regs, need, what in checks:
                waited = 0
                for prev, written, states in reversed(past):
                    if waited >= need:
                        break
                    if prev.startswith(kind) and written & regs:
                        found.append((kernel, text, what))
                    waited += states
        written = set()
        if name.startswith(("s_", "v_")) and operands and not name.startswith(
                ("s_cmp", "s_cbranch", "s_branch", "s_waitcnt", "s_nop", "s_barrier", "s_endpgm")):
            written = _registers(operands[0])
            if len(operands) > 1 and ("_co_" in name or "div_scale" in name):
                written |= _registers(operands[1])
        past = past[-6:] + [(name, written, int(operands[0], 0) + 1 if name == "s_nop" else 1)]
    return copies, found


def test_the_search_itself():
    bad = ["0 <k>:", "\ts_mov_b32 m0, s1", "\tbuffer_load_dwordx4 v1, s[0:3], 0 offen lds"]
    assert hazards(bad) == (1, [("k", bad[2].strip(), "scalar write of M0")])
    assert hazards(bad[:2] + ["\ts_nop 0"] + bad[2:]) == (1, [])
    bad = ["0 <k>:", "\tv_readfirstlane_b32 s2, v1", "\ts_nop 3", "\tbuffer_load_dword v1, v2, s[0:3], 0 offen"]
    assert hazards(bad) == (0, [("k", bad[3].strip(), "VALU write of an SGPR")])
    assert hazards(bad[:2] + ["\ts_nop 4"] + bad[3:]) == (0, [])
    assert hazards(["0 <k>:", "\ts_mov_b32 m0, s1", "\tbuffer_load_dword v1, v2, s[0:3], 0 offen"]) == (0, [])


def test_copies_into_lds_wait_for_their_registers(tmp_path):
    if not os.path.exists(OBJDUMP):
        pytest.skip("llvm-objdump is not installed")
    if not os.path.exists(fb.LIB):
        pytest.fail("libgift.so is not built (python -m fac_whitening_gift_amd.build)")
    shutil.copy(fb.LIB, tmp_path / "libgift.so")
    subprocess.run([OBJDUMP, "--offloading", "libgift.so"], cwd=tmp_path, check=True, capture_output=True)
    objects = sorted(tmp_path.glob("libgift.so.*" + fb.ARCH))
    assert objects
    copies, found = 0, []
    for obj in objects:
        out = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", str(obj)], check=True, capture_output=True,
                             text=True).stdout
        n, bad = hazards(out.splitlines())
        copies += n
        found += bad
    assert copies > 0    # the products' and the covariance's
    assert not found, "%d of %d copies, the first: %s" % (len(found), copies, found[0])
