"""The library and its Python binding are built apart: a host that cannot compile the binding still gets
libzffn.so, and a binding for another torch or Python is neither loaded nor kept."""
import ctypes
import os
import shutil

import pytest
import torch

from quantized_ffn_gb300 import build as zbuild
from quantized_ffn_gb300 import zffn


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """An output folder of its own that holds the compiled objects and nothing linked."""
    zbuild.build()
    for f in os.listdir(zbuild.OUT_DIR):
        if f.endswith(".o"):
            shutil.copy(os.path.join(zbuild.OUT_DIR, f), tmp_path)   # (newer than their sources)
    monkeypatch.setattr(zbuild, "OUT_DIR", str(tmp_path))
    monkeypatch.setattr(zbuild, "LIB", str(tmp_path / "libzffn.so"))
    monkeypatch.setattr(zbuild, "NATIVE", str(tmp_path / "_zffn_native.so"))
    return tmp_path


def compiler(path, text):
    path.write_text("#!/bin/sh\n" + text)
    path.chmod(0o755)
    return str(path)


def test_library_without_the_binding(elsewhere, monkeypatch):
    monkeypatch.setenv("CXX", compiler(elsewhere / "cxx", "echo 'torch/extension.h: no such file' >&2\nexit 1\n"))
    (elsewhere / "_zffn_native.so").write_text("of other sources")
    os.utime(elsewhere / "_zffn_native.so", (0, 0))
    with pytest.warns(RuntimeWarning, match="8-bit and sorting functions are missing"):
        lib = zbuild.build()
    assert ctypes.CDLL(lib).zffn_q4k_row_bytes
    assert not (elsewhere / "_zffn_native.so").exists()


def test_library_where_torch_cannot_be_asked(elsewhere, monkeypatch):
    def no_torch():
        raise ImportError("No module named 'torch'")
    monkeypatch.setattr(zbuild, "_native_command", no_torch)
    with pytest.warns(RuntimeWarning, match="No module named 'torch'"):
        assert os.path.exists(zbuild.build())


def test_binding_is_built_again_for_another_torch(elsewhere, monkeypatch):
    # (the stand-in for the compiler notes its calls and makes the file that it is asked for)
    calls = elsewhere / "calls"
    cxx = compiler(elsewhere / "cxx", f'echo called >> {calls}\nfor a; do out="$a"; done\necho module > "$out"\n')
    monkeypatch.setenv("CXX", cxx)
    count = lambda: len(calls.read_text().split())   # noqa: E731
    zbuild.build()
    assert count() == 1 and (elsewhere / "_zffn_native.so").exists()
    zbuild.build()
    assert count() == 1                               # nothing changed
    monkeypatch.setattr(torch, "__version__", "1.2.3+other")
    zbuild.build()
    assert count() == 2
    zbuild.build()
    assert count() == 2


def test_binding_of_another_torch_is_not_loaded(elsewhere, monkeypatch):
    monkeypatch.setenv("CXX", compiler(elsewhere / "cxx", 'for a; do out="$a"; done\necho no module > "$out"\n'))
    monkeypatch.setattr(torch, "__version__", "1.2.3+other")
    zbuild.build()
    monkeypatch.undo()
    monkeypatch.setattr(zffn, "NATIVE_PATH", str(elsewhere / "_zffn_native.so"))
    monkeypatch.setattr(zffn, "_native_module", None)
    with pytest.raises(RuntimeError, match="1.2.3.*build it again"):
        zffn.moe_sort(torch.zeros((1, 1), dtype=torch.int32), 1)
