"""_bind.so is an addition: without it, or with one for another torch, the
library is built and its calls are made (no GPU needed here)."""
import os
import subprocess

import pytest
import torch

import block_sparse_long_13_b200 as msa
from block_sparse_long_13_b200 import build


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """build's _bind.so in a folder of the test's own."""
    build.build()
    monkeypatch.setattr(build, "BIND", str(tmp_path / "_bind.so"))
    if hasattr(build, "BIND_MADE_FOR"):
        monkeypatch.setattr(build, "BIND_MADE_FOR", str(tmp_path / "_bind.made_for"))
    return tmp_path


def test_the_library_is_built_without_a_compiler_for_bind(elsewhere, monkeypatch, capfd):
    monkeypatch.setenv("CXX", "/nonexistent/g++")
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert "_bind.so was not built" in capfd.readouterr().err
    monkeypatch.setattr(build.subprocess, "run", lambda *a, **k: (_ for _ in ()).throw(subprocess.CalledProcessError(1, "g++")))
    assert build.build() == build.LIB


def test_bind_is_rebuilt_for_another_torch(elsewhere, monkeypatch):
    made = []

    def run(cmd, check):
        made.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
    monkeypatch.setattr(build.subprocess, "run", run)
    build.build()
    build.build()
    assert len(made) == 1 and build.bind_fits()
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    assert not build.bind_fits()
    with pytest.raises(RuntimeError):
        msa._native()
    build.build()
    assert len(made) == 2 and build.bind_fits()


def test_calls_are_made_without_bind(elsewhere, monkeypatch):
    """They reach the same checks by way of Python, and the library by way of ctypes."""
    monkeypatch.setattr(msa, "_calls", None)
    assert not build.bind_fits()
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(msa.MsaError) as e:
        msa.advance_batch(i32(2), i32(2), i32(2, 4), i32(8), i32(4), i32(2), i32(4), i32(3))
    assert "CUDA tensor" in str(e.value)
    monkeypatch.setattr(msa, "_pointers", lambda *a: [16] * (len(a) - 1) + [0])
    monkeypatch.setattr(msa, "_stream_here", lambda s: None)
    with pytest.raises(msa.MsaError) as e:
        msa.advance_batch(i32(2), i32(2), i32(2, 4), i32(8), i32(4), i32(2), i32(4), i32(3), block_size=64)
    assert e.value.status == msa.MSA_ERR_UNSUPPORTED
