"""The kernels' machine code, disassembled: a transfer from memory to LDS takes its target from M0 and needs one wait state
behind an instruction that writes M0. The compiler keeps to that where it writes both; in inline assembly nothing does."""
import os
import re
import shutil
import subprocess

import pytest

import decode_gemm_amd as uw

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"


def _instructions(tmp_path):
    lib = shutil.copy(uw.LIB_PATH, tmp_path / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", lib], check=True, stdout=subprocess.DEVNULL, cwd=tmp_path)
    objects = sorted(f for f in os.listdir(tmp_path) if f.endswith("gfx950"))
    assert objects
    for f in objects:
        p = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", "--no-leading-addr", tmp_path / f], check=True, capture_output=True, text=True)
        yield f, [line.split("//")[0].strip() for line in p.stdout.splitlines() if line.startswith(("\t", " "))]


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no disassembler")
def test_a_transfer_waits_for_m0(tmp_path):
    transfer, writes = re.compile(r"(global_load_lds|buffer_load.*\blds$)"), re.compile(r"s_\w+ m0,")
    seen, bad = 0, []
    for name, code in _instructions(tmp_path):
        for before, now in zip(code, code[1:]):
            if transfer.match(now):
                seen += 1
                if writes.match(before):
                    bad.append(f"{name}: {before}; {now}")
    assert seen > 100
    assert not bad, f"{len(bad)} of {seen} transfers, the first {bad[0]}"
