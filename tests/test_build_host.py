"""What build() does when the CPython extension cannot be compiled (no GPU): the
C library and the dense calls need nvcc alone."""
import ctypes
import os
import shutil
import sysconfig

import pytest

from attention_swa_forward_gb300 import build as B
from attention_swa_forward_gb300 import swa


@pytest.fixture
def small_build(tmp_path, monkeypatch):
    """build() into a folder of its own, of one quick translation unit."""
    monkeypatch.setattr(B, "SOURCES", ["swa_host.cpp"])
    for name in ("BUILD_DIR", "CHECKED_BUILD_DIR"):
        monkeypatch.setattr(B, name, str(tmp_path / name.lower()))
    monkeypatch.setattr(B, "LIB_PATH", str(tmp_path / "libswa.so"))
    monkeypatch.setattr(B, "CHECKED_LIB_PATH", str(tmp_path / "libswa_checked.so"))
    monkeypatch.setattr(B, "PKG", str(tmp_path))  # the extension's folder
    return tmp_path


def failing_compiler(folder, monkeypatch):
    """A g++ that fails on the extension's source alone (as without PyTorch's headers)."""
    folder.mkdir()
    fake = folder / "g++"
    fake.write_text(f'#!/bin/sh\ncase "$*" in *{B.BIND_SOURCE}*) echo no torch headers here >&2; exit 1;; esac\n'
                    f'exec {shutil.which("g++")} "$@"\n')
    fake.chmod(0o755)
    monkeypatch.setenv("PATH", f"{folder}{os.pathsep}{os.environ['PATH']}")


@pytest.mark.parametrize("checked", [False, True])
def test_the_library_is_built_where_the_extension_is_not(small_build, monkeypatch, checked):
    failing_compiler(small_build / "bin", monkeypatch)
    with open(B.bind_path(), "w") as f:
        f.write("of older sources")
    os.utime(B.bind_path(), (1, 1))
    with pytest.warns(RuntimeWarning, match="no torch headers here"):
        path = B.build(checked=checked)
    assert hasattr(ctypes.CDLL(path, mode=os.RTLD_LAZY), "swa_step_host")
    # an extension of older sources is not left to be called
    assert not os.path.exists(B.bind_path())
    # the library is up to date, the extension still missing
    with pytest.warns(RuntimeWarning, match="no torch headers here"):
        assert B.build(checked=checked) == path
    with pytest.raises(RuntimeError, match="no torch headers here"):
        B.build_bind()


def test_both_are_built(small_build):
    assert os.path.exists(B.build())
    assert os.path.getsize(B.bind_path()) > 0 and os.path.dirname(B.bind_path()) == str(small_build)


def test_an_extension_of_another_torch_or_python_is_not_taken(small_build, monkeypatch):
    """It is linked against both, so its file is named after both."""
    torch = pytest.importorskip("torch")
    here = B.bind_path()
    assert torch.__version__ in os.path.basename(here) and here.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    with open(here, "w"):
        pass
    assert not B.is_stale(B.bind_path())
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    assert B.bind_path() != here and B.is_stale(B.bind_path())
    monkeypatch.undo()
    monkeypatch.setattr(sysconfig, "get_config_var", lambda name: ".cpython-399-other.so")
    assert B.bind_path() != here


def test_the_binding_loads_what_build_makes():
    B.build()
    assert swa._bind().__file__ == B.bind_path()
