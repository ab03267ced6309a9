"""The wait states of the attention kernels' own loads to LDS, in the assembly
that the compiler makes of them: a load may read a scalar register that a vector
instruction wrote five states later (it reads the old value before, and with it
memory anywhere), and the compiler does not count states inside an asm block."""
import os
import re
import shutil
import subprocess

import pytest

from chunked_gated_delta_fwd_amd import build

pytestmark = pytest.mark.skipif(shutil.which(build.HIPCC) is None, reason="no hipcc")


def assembly(source, tmp_path):
    flags = [f for f in build.FLAGS if f not in ("-shared", "-fPIC", "-Wall")]
    out = str(tmp_path / "device.s")
    subprocess.run([build.HIPCC] + flags + ["--cuda-device-only", "-S", os.path.join(build.CSRC, source), "-o", out], check=True,
                   stdout=subprocess.DEVNULL, stderr=subprocess.DEVNULL)
    return open(out).read().split("\n")


@pytest.mark.parametrize("source", ["gdr_attn.hip", "gdr_attn_bwd.hip"])
def test_descriptors_are_five_states_old(source, tmp_path):
    lines = [x.strip() for x in assembly(source, tmp_path)]
    lines = [x for x in lines if x and not x.startswith((";", "."))]
    loads = 0
    for i, line in enumerate(lines):
        m = re.match(r"buffer_load_dword(?:x4)? v\d+, s\[(\d+):(\d+)\], 0 offen lds", line)
        if not m:
            continue
        loads += 1
        states = 0
        for back in reversed(lines[max(0, i - 8):i]):
            w = re.match(r"v_(?:readfirstlane|readlane)_b32 s(\d+)", back)
            assert not (w and states < 5 and int(m[1]) <= int(w[1]) <= int(m[2])), (line, back, states)
            n = re.match(r"s_nop (\d+)", back)
            states += int(n[1]) + 1 if n else 1
    assert loads > 50
