"""Wait states that gfx950 leaves to the program, checked in the built library's
own listing.  The compiler inserts them between instructions that it places
itself; inside one inline-assembly string nobody does."""
import os
import re
import shutil
import subprocess

import pytest

from resident_expert_routing_amd import build as _build

OBJDUMP = shutil.which("llvm-objdump") or "/opt/rocm/llvm/bin/llvm-objdump"
TO_LDS = re.compile(r"(global|buffer|scratch)_load_lds_|buffer_load_\w+ .*\blds\b")
WRITES_M0 = re.compile(r"s_\w+ m0\b")


def short_waits(listing: str):
    """(loads to LDS, those right behind an instruction that writes M0).

    A load to LDS takes its LDS address from M0, and one wait state has to pass
    between a scalar write of M0 and the load: any other instruction, s_nop 0
    among them."""
    loads, short, before = 0, [], ""
    for line in listing.splitlines():
        if not line.startswith(("\t", " ")):          # a label or a blank line: another block
            continue
        text = line.split("//")[0].strip()
        if not text:
            continue
        if TO_LDS.match(text):
            loads += 1
            if WRITES_M0.match(before):
                short.append((before, text))
        before = text
    return loads, short


def test_the_check_finds_what_it_looks_for():
    good = "<k>:\n\ts_mov_b32 m0, s2\n\ts_nop 0 // 1\n\tglobal_load_lds_dwordx4 v[2:3], off // 2\n"
    bad = "<k>:\n\ts_mov_b32 m0, s2 // 0\n\tglobal_load_lds_dwordx4 v[2:3], off nt // 1\n"
    assert short_waits(good) == (1, [])
    assert short_waits(bad)[0] == 1 and len(short_waits(bad)[1]) == 1
    assert len(short_waits(bad.replace("global_load_lds_dwordx4 v[2:3], off nt",
                                       "buffer_load_dword v2, s[4:7], 0 offen lds"))[1]) == 1


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no llvm-objdump")
def test_loads_to_lds_wait_for_m0(tmp_path):
    lib = tmp_path / "lib.so"
    shutil.copy(_build.LIB, lib)
    subprocess.run([OBJDUMP, "--offloading", str(lib)], check=True, capture_output=True,
                   cwd=tmp_path, timeout=120)
    parts = sorted(p for p in os.listdir(tmp_path) if p.endswith("gfx950"))
    assert parts, "no device code in the library"
    loads, short = 0, []
    for part in parts:
        r = subprocess.run([OBJDUMP, "-d", str(tmp_path / part)], check=True, capture_output=True,
                           text=True, timeout=120)
        n, s = short_waits(r.stdout)
        loads, short = loads + n, short + s
    assert loads > 0
    assert not short, f"{len(short)} of {loads} loads to LDS follow their M0 at once: {short[0]}"
