"""Build ``libgdr.so`` (HIP kernels + C ABI) for gfx950 with hipcc, and
``_gdr_torch.so`` (the compiled marshalling of mixer.py and attention.py), in-tree."""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libgdr.so")
TORCH_LIB = os.path.join(PKG, "_gdr_torch.so")

SOURCES = ["gdr_kernels.hip", "gdr_bwd.hip", "gdr_kda.hip", "gdr_conv.hip", "gdr_qknorm.hip", "gdr_ssm.hip",
           "gdr_ssm_bwd.hip", "gdr_attn.hip", "gdr_attn_bwd.hip", "gdr_paged.hip", "gdr_api.cpp", "gdr_mixer_api.cpp",
           "gdr_attn_api.cpp"]

ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
HIPCC = os.environ.get("HIPCC", os.path.join(ROCM, "bin", "hipcc"))

FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++20",
    "-fPIC",
    "-shared",
    "-Wall",
    "-Wno-unused-function",
    # keep the compiler from emitting packed fp32 (v_pk_*_f32) instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", INCLUDE,
    "-I", CSRC,
]


def _torch_command() -> list:
    """The host compiler's line for the extension that mixer.py calls; raises
    ImportError where torch, its headers or a host compiler are missing."""
    import torch
    from torch.utils import cpp_extension

    root = os.path.dirname(torch.__file__)
    paths = cpp_extension.include_paths()
    if not any(os.path.exists(os.path.join(p, "torch", "extension.h")) for p in paths):
        raise ImportError("torch's headers are not installed")
    if shutil.which("g++") is None:
        raise ImportError("g++ was not found")
    include = sum((["-isystem", p] for p in paths), [])
    return (["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
             "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI), "-DTORCH_EXTENSION_NAME=_gdr_torch"]
            + include + ["-isystem", os.path.join(ROCM, "include"), "-isystem", sysconfig.get_paths()["include"], "-I", INCLUDE,
                         os.path.join(CSRC, "gdr_torch.cpp"), "-L", os.path.join(root, "lib"), "-lc10", "-lc10_hip", "-ltorch_cpu",
                         "-ltorch", "-ltorch_python", "-L", PKG, "-lgdr", "-Wl,-rpath,$ORIGIN"])


def build(verbose: bool = False) -> str:
    """Compile every source into ``chunked_gated_delta_fwd_amd/libgdr.so``, then
    the torch extension that links to it.  The C ABI does not need the
    extension: without torch, its headers or g++ the library is built alone, and
    mixer.py says what is missing when it is imported."""
    _compile([HIPCC] + FLAGS + [os.path.join(CSRC, s) for s in SOURCES], LIB, verbose)
    try:
        command = _torch_command()
    except ImportError as e:
        if os.path.exists(TORCH_LIB):   # of other sources
            os.remove(TORCH_LIB)
        print("_gdr_torch.so is not built (%s): the Python calls of mixer.py need it" % e, file=sys.stderr, flush=True)
        return LIB
    _compile(command, TORCH_LIB, verbose)
    return LIB


def _compile(cmd: list, lib: str, verbose: bool) -> None:
    tmp = lib + ".tmp%d" % os.getpid()
    cmd = cmd + ["-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    proc = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    out = "\n".join(line for line in proc.stdout.splitlines()
                    if "packed-fp32-ops" not in line and line.strip())
    if proc.returncode != 0:
        if os.path.exists(tmp):
            os.remove(tmp)
        raise RuntimeError("%s failed (%d):\n%s" % (os.path.basename(cmd[0]), proc.returncode, out))
    if verbose and out:
        print(out, flush=True)
    os.replace(tmp, lib)


if __name__ == "__main__":
    build(verbose="-v" in sys.argv)
    print(LIB)
