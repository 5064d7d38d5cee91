"""Wait states in the built GPU code (no GPU needed).  The compiler keeps the
wait states of gfx950 between the instructions that it schedules, but not
inside or next to inline assembly.  The disassembly of the library is searched
for the two rules that its assembly has to keep by itself:

* a copy to LDS needs one wait state after a scalar write of M0 (its LDS address);
* a vector memory instruction needs five after a vector instruction wrote one
  of its scalar registers.
"""

import glob
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OBJDUMP = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin", "llvm-objdump")
SCALAR = re.compile(r"\bs\[(\d+):(\d+)\]|\bs(\d+)\b|\b(vcc|m0)\b")
VECTOR_MEMORY = ("buffer_", "global_", "flat_", "scratch_")
# vector instructions whose second operand is a scalar result too (a carry)
TWO_RESULTS = re.compile(r"v_(add|sub|subrev|addc|subb|subbrev)_co_|v_mad_[iu]64|v_div_scale")


def _scalars(text):
    out = set()
    for lo, hi, one, name in SCALAR.findall(text):
        out |= set(range(int(lo), int(hi) + 1)) if lo else {int(one)} if one else {name}
    return out


def hazards(lines):
    """([instruction, wait states, needed], copies to LDS seen) of a disassembly
    in the order of its addresses."""
    found, copies, at, m0, written = [], 0, 0, None, {}
    for line in lines:
        text = line.split("//")[0].strip()
        if text.endswith(">:"):   # another function
            m0, written = None, {}
            continue
        op, _, rest = text.partition(" ")
        if not re.match(r"[a-z]+_", op):
            continue
        args = rest.split(",")
        if op == "s_nop":
            at += int(args[0], 0) + 1
            continue
        if op.startswith(VECTOR_MEMORY):
            if "_lds_" in op or text.endswith(" lds"):
                copies += 1
                if m0 is not None and at - m0 - 1 < 1:
                    found.append((text, at - m0 - 1, 1))
            for r in _scalars(rest):
                if r in written and at - written[r] - 1 < 5:
                    found.append((text, at - written[r] - 1, 5))
        elif op.startswith("v_"):
            for r in _scalars(args[0]) | (_scalars(args[1]) if len(args) > 1 and TWO_RESULTS.match(op) else set()):
                written[r] = at
        elif op.startswith("s_"):
            for r in _scalars(args[0]):
                written.pop(r, None)
                m0 = at if r == "m0" else m0
        at += 1
    return found, copies


def test_the_search_finds_what_it_looks_for():
    near = ["<f>:", "s_mov_b32 m0, s4", "buffer_load_dwordx4 v1, s[8:11], 0 offen lds"]
    assert hazards(near) == ([(near[2], 0, 1)], 1)
    assert hazards(near[:2] + ["s_nop 0"] + near[2:]) == ([], 1)
    near = ["<f>:", "v_readfirstlane_b32 s9, v3", "s_nop 3", "buffer_load_dword v1, v2, s[8:11], 0 offen"]
    assert hazards(near) == ([(near[3], 4, 5)], 0)
    assert hazards(near[:2] + ["s_nop 4"] + near[3:]) == ([], 0)
    assert hazards(near[:2] + ["s_mov_b32 s9, 0"] + near[3:]) == ([], 0)


def test_wait_states_of_the_built_library(tmp_path):
    if not os.path.exists(OBJDUMP):
        pytest.skip("llvm-objdump not available")
    lib = shutil.copy(os.path.join(ROOT, "fp8_block_scaled_dsmoe_amd", "libdsmoe.so"), tmp_path)
    subprocess.run([OBJDUMP, "--offloading", lib], cwd=tmp_path, check=True, capture_output=True)
    images = glob.glob(os.path.join(tmp_path, "*gfx950"))
    assert images
    found, copies = [], 0
    for image in images:
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", "--no-leading-addr", image], check=True,
                              capture_output=True, text=True).stdout
        f, c = hazards(text.splitlines())
        found += f
        copies += c
    assert copies > 100, "the copies to LDS are not recognised"
    assert not found, f"{len(found)} places, first {found[:3]}"
