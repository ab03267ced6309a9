"""The attention kernels' own loads to LDS write m0 in their asm block: the block
says so to the compiler, which uses that register for itself where it likes, and
in the assembly each load has its write of m0 and its wait directly before it,
whatever branches there, with no other use of m0 in the file."""
import os
import re
import shutil
import subprocess

import pytest

from chunked_gated_delta_fwd_amd import build
from test_attn_waits import assembly

pytestmark = pytest.mark.skipif(shutil.which(build.HIPCC) is None, reason="no hipcc")

SOURCES = ["gdr_attn.hip", "gdr_attn_bwd.hip"]


@pytest.mark.parametrize("source", SOURCES)
def test_the_compiler_is_told(source, tmp_path):
    flags = [f for f in build.FLAGS if f not in ("-shared", "-fPIC", "-Wall", "-O3")]
    out = str(tmp_path / "device.ll")
    subprocess.run([build.HIPCC] + flags + ["-O1", "-Xclang", "-disable-llvm-passes", "--cuda-device-only", "-S", "-emit-llvm",
                                            os.path.join(build.CSRC, source), "-o", out],
                   check=True, stdout=subprocess.DEVNULL, stderr=subprocess.DEVNULL)
    blocks = re.findall(r'asm sideeffect "([^"]*)", "([^"]*)"', open(out).read())
    loads = [constraints for text, constraints in blocks if "m0" in text]
    assert loads and all("~{m0}" in c.split(",") for c in loads), loads


@pytest.mark.parametrize("source", SOURCES)
def test_each_load_has_its_own_write_and_wait(source, tmp_path):
    lines = [x.strip() for x in assembly(source, tmp_path)]
    lines = [x for x in lines if x and not x.startswith((";", "."))]
    loads = [i for i, x in enumerate(lines) if re.match(r"buffer_load_dword(x4)? .* lds$", x)]
    for i in loads:
        wait = re.fullmatch(r"s_nop (\d+)", lines[i - 1])
        assert wait and int(wait[1]) >= 4 and lines[i - 2].startswith("s_mov_b32 m0, "), lines[i - 2:i + 1]
    assert len(loads) > 50
    assert sum(bool(re.search(r"\bm0\b", x)) for x in lines) == len(loads)
