"""The wait states that loads from global memory to LDS need, in the machine
code of this library as it was built from its sources.

The loads are issued from inline assembly, in which the compiler inserts no
wait states.  For this family of processors the instruction set asks for
  * 1 wait state between a scalar instruction that writes M0 and a load to LDS
    (which takes its LDS address from M0), and
  * 5 between a vector instruction that writes a scalar register and a memory
    instruction that reads that register.
Each instruction is one wait state, s_nop n is n + 1.
"""
import glob
import os
import re
import shutil
import subprocess

import pytest

import gemm_rbq_encode_amd as rbq

OBJDUMP = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin", "llvm-objdump")


def registers(operand):
    """Scalar registers of an operand (s5, s[4:5], m0, vcc)."""
    m = re.fullmatch(r"s\[(\d+):(\d+)\]", operand)
    if m:
        return set(range(int(m[1]), int(m[2]) + 1))
    m = re.fullmatch(r"s(\d+)", operand)
    if m:
        return {int(m[1])}
    return {operand} if operand in ("m0", "vcc") else set()


def short_waits(lines):
    """(number of loads to LDS, [(function, instructions before, load)] of those that come too early)."""
    loads, bad, where, before = 0, [], "?", []
    for line in lines:
        m = re.match(r"[0-9a-f]+ <(.*)>:", line)
        if m:
            where, before = m[1], []
            continue
        text = line.split("//")[0].strip()
        op, _, rest = text.partition(" ")
        args = [a.split()[0] for a in rest.split(",") if a.split()]
        if re.match(r"global_load_lds|scratch_load_lds", op) or (op.startswith("buffer_load") and rest.split()[-1:] == ["lds"]):
            loads += 1
            read = set().union(*[registers(a) for a in args])
            waited = 0
            for o, a in reversed(before):
                written = registers(a[0]) if a else set()
                if (waited < 1 and o.startswith("s_") and "m0" in written) or \
                        (waited < 5 and o.startswith("v_") and written & (read | {"m0"})):
                    bad.append((where, [b[0] for b in before[-3:]], text))
                waited += int(a[0], 0) + 1 if o == "s_nop" else 1
                if waited >= 5:
                    break
        if op:
            before = (before + [(op, args)])[-6:]
    return loads, bad


def test_the_scan_finds_what_it_is_for():
    code = ["0000 <k>:", "s_mov_b32 m0, s3", "global_load_lds_dwordx4 v0, s[0:1]"]
    assert short_waits(code) == (1, [("k", ["s_mov_b32"], code[2])])
    assert short_waits(code[:2] + ["s_nop 0"] + code[2:]) == (1, [])
    code = ["0000 <k>:", "v_readfirstlane_b32 s1, v4", "s_mov_b32 m0, s3", "s_nop 2", "global_load_lds_dword v0, s[0:1]"]
    assert len(short_waits(code)[1]) == 1
    code[3] = "s_nop 3"
    assert short_waits(code) == (1, [])


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no llvm-objdump")
def test_every_load_to_lds_waits_for_its_address(tmp_path):
    lib = shutil.copy(rbq.LIB_PATH, tmp_path)
    subprocess.run([OBJDUMP, "--offloading", lib], cwd=tmp_path, check=True, capture_output=True, timeout=60)
    total = 0
    for f in sorted(glob.glob(os.path.join(tmp_path, "*gfx950*"))):
        out = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", f], check=True, capture_output=True, text=True,
                             timeout=60).stdout
        loads, bad = short_waits(out.splitlines())
        total += loads
        assert not bad, f"{len(bad)} loads too early, e.g. {bad[0]}"
    assert total > 0                     # the library has such loads
