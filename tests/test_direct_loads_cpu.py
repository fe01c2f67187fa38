"""Loads from memory straight to LDS in the built kernels: their asm statements are closed to
the compiler's hazard pass, so the wait states that the instructions need are looked for in the
disassembly of what was built."""

import os
import re
import shutil
import struct
import subprocess

import pytest

from segmented_gather_gemm_lora_amd import binding as B

MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


def code_objects(path):
    """The gfx950 code objects of a library."""
    raw = open(path, "rb").read()
    at = raw.find(MAGIC)
    while at >= 0:
        count, = struct.unpack_from("<Q", raw, at + len(MAGIC))
        entry = at + len(MAGIC) + 8
        for _ in range(count):
            offset, size, length = struct.unpack_from("<QQQ", raw, entry)
            triple = raw[entry + 24: entry + 24 + length].decode()
            entry += 24 + length
            if "gfx950" in triple and size:
                yield raw[at + offset: at + offset + size]
        at = raw.find(MAGIC, at + len(MAGIC))


def scalars(operand):
    """Numbers of the scalar registers that an operand names."""
    m = re.fullmatch(r"s(\d+)|s\[(\d+):(\d+)\]", operand.strip())
    if not m:
        return set()
    return {int(m[1])} if m[1] else set(range(int(m[2]), int(m[3]) + 1))


def states(line):
    """Wait states that an instruction is worth to those behind it."""
    return int(line.split()[1], 0) + 1 if line.startswith("s_nop") else 1


def before(lines, at, wanted):
    """The instructions less than `wanted` wait states before instruction `at`."""
    passed = 0
    while at > 0 and passed < wanted:
        at -= 1
        yield lines[at]
        passed += states(lines[at])


def faults(lines):
    """Loads to LDS in a listing, and those that come too soon: one wait state behind a scalar
    write of m0, five behind a vector instruction's write of their scalar address."""
    loads, bad = 0, []
    for i, line in enumerate(lines):
        if "global_load_lds" not in line:
            continue
        loads += 1
        address = set().union(*(scalars(o) for o in line.split(None, 1)[1].split(" offset")[0].split(",")))
        if any(re.match(r"s_\w+ m0\b", p) for p in before(lines, i, 1)):
            bad.append(("m0", line))
        for p in before(lines, i, 5):
            if p.startswith("v_") and " " in p:
                written = p.split(None, 1)[1].split(",")[: 2 if re.match(r"v_\w*(_co_|div_scale)", p) else 1]
                if address & set().union(*map(scalars, written)):
                    bad.append((p, line))
    return loads, bad


def test_the_search_finds_both():
    ok = ["v_readlane_b32 s4, v1, 3", "s_mov_b32 m0, s7", "s_nop 3", "global_load_lds_dwordx4 v2, s[4:5]"]
    assert faults(ok) == (1, [])
    assert len(faults([ok[0], ok[1], "s_nop 0", ok[3]])[1]) == 1
    assert len(faults([ok[1], ok[3]])[1]) == 1
    assert faults([ok[1], "v_add_u32_e32 v2, v2, v3", ok[3]]) == (1, [])


def test_wait_states(tmp_path):
    objdump = shutil.which("llvm-objdump") or "/opt/rocm/llvm/bin/llvm-objdump"
    if not os.path.exists(objdump):
        pytest.skip("no llvm-objdump")
    total = 0
    for i, code in enumerate(code_objects(B.lib_path())):
        elf = tmp_path / f"{i}.elf"
        elf.write_bytes(code)
        text = subprocess.run([objdump, "-d", "--no-show-raw-insn", str(elf)], capture_output=True, text=True, check=True).stdout
        lines = [t for t in (ln.split("//")[0].strip() for ln in text.splitlines()) if t]
        loads, bad = faults(lines)
        assert not bad, f"{len(bad)} of {loads}, first: {bad[0]}"
        total += loads
    assert total > 0
