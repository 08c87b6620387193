"""Wait states that gfx950 leaves to the program, in the library's own device
code.  The compiler keeps them between the instructions it emits, and cannot
inside an asm block; nothing on the GPU shows a missing one reliably.

 - M0 written by a scalar instruction, then read by a load to LDS: 1.
 - An SGPR written by a vector instruction, then read by a vector memory
   instruction: 5.
Each instruction is one wait state, s_nop N is N + 1.
"""
import os
import re
import shutil
import subprocess

import pytest

from bit_moe_amd import _lib

OBJDUMP = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin", "llvm-objdump")
VMEM = re.compile(r"(global|buffer|flat|scratch)_")
SGPR = re.compile(r"\bs(?:(\d+)\b|\[(\d+):(\d+)\])|\b(vcc)(?:_lo|_hi)?\b")
# vector instructions whose second operand is written too (a carry, or a flag)
SECOND = re.compile(r"v_(\w*_co_|mad_u64_u32|mad_i64_i32|div_scale_)")


def sgprs(text):
    out = set()
    for one, lo, hi, vcc in SGPR.findall(text):
        out |= {"vcc"} if vcc else {int(one)} if one else set(range(int(lo), int(hi) + 1))
    return out


def missing(lines):
    """(line number, text, what is missing) of each such place."""
    found, now, m0_at, at = [], 0, -9, {}
    for number, line in enumerate(lines):
        op, _, rest = line.strip().partition(" ")
        if line.endswith(">:"):                              # a function
            now, m0_at, at = now + 9, -9, {}
            continue
        if not rest and not op.startswith("s_"):
            continue
        args = rest.split("//")[0].split(",")
        if VMEM.match(op):
            if ("_load_lds" in op or args[-1].rstrip().endswith(" lds")) and now - m0_at < 2:
                found.append((number, line.strip(), "M0"))
            if any(now - at.get(r, -9) < 6 for r in sgprs(rest)):
                found.append((number, line.strip(), "SGPR"))
        elif op.startswith("v_"):
            writes = sgprs(args[0]) | (sgprs(args[1]) if SECOND.match(op) and len(args) > 1 else set())
            if op.startswith("v_cmp") and op.endswith("_e32"):
                writes.add("vcc")
            for r in writes:
                at[r] = now
        elif op.startswith("s_"):
            if args[0].strip() == "m0":
                m0_at = now
            if op == "s_nop":
                now += int(args[0], 0)
        now += 1
    return found


def test_the_scan_sees_what_is_missing():
    ok = ["s_mov_b32 m0, s1", "s_nop 0", "global_load_lds_dwordx4 v[2:3], off"]
    assert not missing(ok) and [f[2] for f in missing([ok[0], ok[2]])] == ["M0"]
    assert not missing([ok[0], "v_mov_b32_e32 v0, v1", ok[2]])
    read = ["v_readlane_b32 s4, v40, 3", "s_mov_b32 m0, s1", "s_nop 0", "global_load_lds_dwordx4 v2, s[4:5]"]
    assert [f[2] for f in missing(read)] == ["SGPR"]
    assert not missing(read[:2] + ["s_nop 3"] + read[3:]) and missing(read[:2] + ["s_nop 2"] + read[3:])
    assert not missing([read[0], "s_mov_b64 s[6:7], s[4:5]", *read[1:3], "global_load_lds_dwordx4 v2, s[6:7]"])
    assert [f[2] for f in missing(["v_cmp_lt_u32_e64 s[8:9], v0, v1", "global_load_dword v0, v1, s[8:9]"])] == ["SGPR"]
    assert [f[2] for f in missing(["v_add_co_u32_e64 v0, s[8:9], v0, v1", "buffer_load_dword v0, v1, s[8:11], 0 offen lds"])] \
        == ["SGPR"]


def test_library_keeps_the_wait_states(tmp_path):
    if not os.path.exists(OBJDUMP) or not os.path.exists(_lib.LIB_PATH):
        pytest.skip("needs the built library and llvm-objdump")
    lib = shutil.copy(_lib.LIB_PATH, tmp_path)
    subprocess.run([OBJDUMP, "--offloading", lib], check=True, cwd=tmp_path, stdout=subprocess.DEVNULL)
    code = sorted(str(p) for p in tmp_path.iterdir() if p.name.endswith("gfx950") and p.stat().st_size)
    assert code
    lines = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", "--no-leading-addr", *code], check=True,
                           capture_output=True, text=True).stdout.splitlines()
    found = missing(lines)
    assert sum("_load_lds" in line for line in lines) > 1000
    assert not found, f"{len(found)} places, the first {found[:3]}"
