"""Wait states around the copies from memory to LDS, in the built library.

The copies are written in inline assembly, where the compiler inserts no wait
states of its own:

  - an instruction that writes M0 (the LDS address) is not directly followed
    by the copy that uses it: one wait state is needed;
  - between a vector instruction that writes a scalar register (a lane read, a
    comparison) and a copy whose base that register holds, five are needed.

Every instruction is a wait state, s_nop N is N + 1.  The library's own code is
disassembled for this; no GPU is needed.
"""

import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "post_pruning_amd", "libsg.so")
OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"

pytestmark = pytest.mark.skipif(not (os.path.exists(OBJDUMP) and os.path.exists(LIB)),
                                reason="llvm-objdump or libsg.so missing")

COPY = re.compile(r"^(global_load_lds_dword\w*|buffer_load_dword\w* .*\blds\b)")
SGPRS = re.compile(r"\bs\[(\d+):(\d+)\]|\bs(\d+)\b|\b(vcc)\b")


def _scalars(operand):
    out = set()
    for lo, hi, one, vcc in SGPRS.findall(operand):
        if vcc:
            out.add("vcc")
        elif one:
            out.add(int(one))
        else:
            out.update(range(int(lo), int(hi) + 1))
    return out


def hazards(lines):
    """(copies, [(what, text)]) of one kernel's instructions, as text."""
    found, copies, last = [], 0, []  # last: (instruction, wait states since the one before it began)
    for text in lines:
        if COPY.match(text):
            copies += 1
            ops = text.split(None, 1)[1].split(",")
            base = set().union(*(_scalars(o) for o in ops))
            waited = 0
            for prev in reversed(last):
                name, _, rest = prev.partition(" ")
                if name == "s_nop":
                    waited += int(rest.split()[0], 0) + 1
                    continue
                dst = rest.split(",")[0].strip()
                if dst == "m0" and waited < 1:
                    found.append(("M0", f"{prev} / {text}"))
                if name.startswith("v_") and waited < 5 and _scalars(dst) & base:
                    found.append(("base", f"{prev} / {text}"))
                waited += 1
                if waited >= 5:
                    break
        last.append(text)
        del last[:-8]
    return copies, found


def test_the_check_itself():
    copy = "global_load_lds_dwordx4 v2, s[10:11]"
    assert hazards(["s_mov_b32 m0, s30", copy])[1]
    assert not hazards(["s_mov_b32 m0, s30", "s_nop 0", copy])[1]
    assert not hazards(["s_mov_b32 m0, s30", "v_add_u32_e32 v1, v2, v3", copy])[1]
    assert hazards(["v_readlane_b32 s11, v9, 3", "s_mov_b32 m0, s30", "s_nop 0", copy])[1]
    assert hazards(["v_cmp_lt_i64_e64 s[10:11], v[2:3], v[4:5]", "s_nop 3", copy])[1]
    assert not hazards(["v_readlane_b32 s11, v9, 3", "s_nop 4", copy])[1]
    assert not hazards(["v_readlane_b32 s12, v9, 3", "s_mov_b32 m0, s30", "s_nop 0", copy])[1]
    assert hazards([copy])[0] == 1


def test_waits_of_every_copy(tmp_path):
    lib = str(tmp_path / "libsg.so")
    shutil.copy(LIB, lib)
    subprocess.run([OBJDUMP, "--offloading", lib], check=True, capture_output=True, cwd=tmp_path)
    objects = sorted(f for f in os.listdir(tmp_path) if f.endswith("gfx950"))
    assert objects
    total, found = 0, []
    for obj in objects:
        res = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", str(tmp_path / obj)], check=True,
                             capture_output=True, text=True)
        if "load_lds" not in res.stdout and " lds" not in res.stdout:
            continue
        kernel, lines = None, []
        for line in res.stdout.splitlines() + ["0 <end>:"]:
            head = re.match(r"^[0-9a-f]+ <(.*)>:$", line)
            if head:
                copies, bad = hazards(lines)
                total += copies
                found += [(kernel, *b) for b in bad]
                kernel, lines = head.group(1), []
            elif line.startswith("\t"):
                lines.append(line.split("//")[0].strip())
    assert total > 100, "no copies found"
    assert not found, f"{len(found)} of {total} copies: {found[:3]}"
