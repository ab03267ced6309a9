"""What build() does where the torch extension cannot be built: the library alone."""
import os
import sys

import pytest

from chunked_gated_delta_fwd_amd import build


@pytest.fixture
def compiled(monkeypatch, tmp_path):
    """build() with the compilers' calls written down instead of made."""
    done = []
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libgdr.so"))
    monkeypatch.setattr(build, "TORCH_LIB", str(tmp_path / "_gdr_torch.so"))
    monkeypatch.setattr(build, "_compile", lambda cmd, lib, verbose: done.append((cmd[0], os.path.basename(lib))))
    return done


def test_library_then_extension(compiled):
    assert build.build() == build.LIB
    assert compiled == [(build.HIPCC, "libgdr.so"), ("g++", "_gdr_torch.so")]


@pytest.mark.parametrize("missing", ["torch", "headers", "g++"])
def test_library_alone(compiled, monkeypatch, capsys, missing):
    if missing == "torch":
        monkeypatch.setitem(sys.modules, "torch", None)
    elif missing == "headers":
        from torch.utils import cpp_extension
        monkeypatch.setattr(cpp_extension, "include_paths", lambda *a, **k: ["/nowhere"])
    else:
        monkeypatch.setattr("shutil.which", lambda *a, **k: None)
    open(build.TORCH_LIB, "w").close()   # of an earlier build
    assert build.build() == build.LIB
    assert compiled == [(build.HIPCC, "libgdr.so")]
    assert not os.path.exists(build.TORCH_LIB) and "_gdr_torch.so is not built" in capsys.readouterr().err
