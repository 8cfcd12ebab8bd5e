"""The build without a host C++ compiler, as with hipcc alone (the HIP sources are not compiled here)."""
import os
import shutil
import subprocess
import sys

import pytest

from w4a16_routed_expert_moe_amd import build as b


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """The build's outputs under tmp_path, its HIP objects and their link replaced."""
    monkeypatch.setattr(b, "BUILD_DIR", str(tmp_path))
    monkeypatch.setattr(b, "LIB_PATH", str(tmp_path / "libmoe_w4a16.so"))
    monkeypatch.setattr(b, "BIND_PATH", str(tmp_path / "_bind.so"))
    monkeypatch.setattr(b, "_compile", lambda src: src)
    real = subprocess.run

    def run(cmd, **kw):
        if cmd[0] != b.HIPCC:
            return real(cmd, **kw)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(subprocess, "run", run)
    return tmp_path


@pytest.mark.parametrize("cxx", ["false", "no-such-compiler", "false --flag"])
def test_without_a_host_compiler(elsewhere, monkeypatch, cxx):
    """The library is built all the same, and no native checks of an earlier build stay beside it."""
    monkeypatch.setenv("CXX", cxx)
    (elsewhere / "_bind.so").write_bytes(b"of an earlier build")
    with pytest.warns(UserWarning, match="checked in Python"):
        assert b.build() == b.LIB_PATH
    assert os.path.exists(b.LIB_PATH) and not os.path.exists(b.BIND_PATH)
    assert not [f for f in os.listdir(elsewhere) if f.startswith("_bind")]


def test_without_the_headers_of_torch(elsewhere, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch.utils.cpp_extension", None)  # importing it fails
    with pytest.warns(UserWarning, match="checked in Python"):
        b.build()
    assert os.path.exists(b.LIB_PATH) and not os.path.exists(b.BIND_PATH)


@pytest.mark.skipif(not shutil.which("g++"), reason="g++ not found")
def test_with_one(elsewhere, monkeypatch, recwarn):
    monkeypatch.delenv("CXX", raising=False)
    b.build()
    assert os.path.exists(b.LIB_PATH) and os.path.getsize(b.BIND_PATH) > 10000
    assert not [w for w in recwarn if "_bind" in str(w.message)]
