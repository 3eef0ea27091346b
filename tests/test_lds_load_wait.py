"""A load into LDS takes its LDS address from M0, and reads the old value when it is the very
next instruction after a scalar write of M0: one wait state has to lie between.  The compiler
sees to it for its own loads, not inside an inline-assembly string, so the built library is
looked through (host only; the code objects are those compiled here)."""
import os
import re
import shutil
import subprocess

import pytest

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
INSTR = re.compile(r"^\t(\S+)(?:\s+(.*?))?\s*//")


def unwaited(lines):
    """(loads into LDS through M0, those right behind a scalar write of M0)."""
    loads, bad, prev = 0, [], ("", "")
    for line in lines:
        m = INSTR.match(line)
        if not m:
            continue   # labels and headers: a branch target does not move the instruction before it
        op, args = m.group(1), m.group(2) or ""
        if "_load_lds_" in op or (op.startswith("buffer_load") and re.search(r"\blds\b", args)):
            loads += 1
            if prev[0].startswith("s_") and re.match(r"m0\b", prev[1]):
                bad.append(f"{prev[0]} {prev[1]}; {op} {args}")
        prev = (op, args)
    return loads, bad


def test_the_search_itself():
    write, nop, load = "\ts_mov_b32 m0, s4    // 0: 1\n", "\ts_nop 0    // 4: 1\n", \
        "\tglobal_load_lds_dwordx4 v[0:1], off    // 8: 1\n"
    assert unwaited([write, nop, load]) == (1, [])
    assert len(unwaited([write, load])[1]) == 1
    assert len(unwaited([write, "0000 <L1>:\n", load])[1]) == 1
    assert unwaited([load, write]) == (1, [])


def test_a_wait_state_between_m0_and_the_load(tmp_path):
    from combine_top_router_amd import lib as L
    if not os.path.exists(L.lib_path()) or not os.path.exists(OBJDUMP):
        pytest.skip("libmoe.so or llvm-objdump not there")
    so = shutil.copy(L.lib_path(), tmp_path)
    subprocess.run([OBJDUMP, "--offloading", so], cwd=tmp_path, check=True, capture_output=True)
    objs = [p for p in tmp_path.iterdir() if p.name.endswith("gfx950")]
    assert objs
    loads = 0
    for p in objs:
        with subprocess.Popen([OBJDUMP, "-d", str(p)], stdout=subprocess.PIPE, text=True) as d:
            n, bad = unwaited(d.stdout)
        assert d.returncode == 0
        assert not bad, (len(bad), bad[:3])
        loads += n
    assert loads > 100   # the GEMMs' rings
