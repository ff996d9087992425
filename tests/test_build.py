"""The build of the host module: what happens where it cannot be built (no GPU needed)."""

import os
import subprocess
import sys

import pytest

from gguf_quant_matmul_amd import build


@pytest.mark.parametrize("missing", ["torch", "compiler", "headers"])
def test_without_its_needs_the_host_module_is_left_out(monkeypatch, tmp_path, missing):
    call = tmp_path / "_kqcall.so"
    call.write_bytes(b"of an earlier build")
    monkeypatch.setattr(build, "CALL", str(call))
    if missing == "torch":
        monkeypatch.setitem(sys.modules, "torch", None)
    elif missing == "compiler":
        monkeypatch.setattr(build.shutil, "which", lambda name: str(tmp_path / "no-such-compiler"))
    else:
        run = subprocess.run
        monkeypatch.setattr(build.subprocess, "run", lambda cmd, **kw: run(
            [sys.executable, "-c", "import sys; sys.exit('Python.h: No such file')"], **kw))
    with pytest.warns(RuntimeWarning, match="_kqcall.so is not built"):
        build._call_module(verbose=False, incremental=False)
    assert os.listdir(tmp_path) == []
