"""The build without compilers: stand-ins for nvcc and the host compiler write the
files they are asked for, so that what is built, in which order and under which
name can be seen in a folder of its own."""
import os
import stat
import sys
import sysconfig

import pytest

from gated_delta_rule_varlen_gb300 import build


def script(path, text):
    path.write_text("#!/bin/sh\n" + text)
    path.chmod(path.stat().st_mode | stat.S_IXUSR)
    return str(path)


WRITES = 'while [ $# -gt 0 ]; do if [ "$1" = -o ]; then echo made > "$2"; fi; shift; done\n'


@pytest.fixture
def folder(tmp_path, monkeypatch):
    monkeypatch.setattr(build, "LIBDIR", str(tmp_path / "lib"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "lib" / "libgdr.so"))
    (tmp_path / "bin").mkdir()
    compiler = script(tmp_path / "bin" / "nvcc", WRITES)
    monkeypatch.setattr(build, "nvcc", lambda: compiler)
    monkeypatch.setenv("CXX", script(tmp_path / "cxx", WRITES))
    return tmp_path


def made(folder):
    return sorted(f for f in os.listdir(folder / "lib") if f.endswith(".so"))


def test_library_and_binding(folder):
    import torch
    assert build.build() == str(folder / "lib" / "libgdr.so")
    # compiled against one PyTorch and one Python: both are in its name
    name = f"_gdr_ops-{torch.__version__}.{sysconfig.get_config_var('SOABI')}.so"
    assert made(folder) == sorted([name, "libgdr.so"]) and build.binding_path() == str(folder / "lib" / name)
    assert f"cpython-{sys.version_info[0]}{sys.version_info[1]}" in name
    assert not [f for f in os.listdir(folder / "lib") if ".tmp" in f]


def test_library_alone_without_pytorch(folder, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)  # importing it raises ImportError
    build.build()
    assert made(folder) == ["libgdr.so"] and "PyTorch" in capsys.readouterr().err


def test_library_is_linked_before_an_error_in_the_binding(folder, monkeypatch):
    monkeypatch.setenv("CXX", script(folder / "broken", "echo no such header; exit 1\n"))
    with pytest.raises(RuntimeError, match="gdr_binding.cpp:\\nno such header"):
        build.build()
    assert made(folder) == ["libgdr.so"]


def test_an_error_in_a_kernel_links_nothing(folder, monkeypatch):
    compiler = script(folder / "bin" / "nvcc", 'case "$*" in *gdr_step.cu*) echo bad kernel; exit 1;; esac\n' + WRITES)
    monkeypatch.setattr(build, "nvcc", lambda: compiler)
    with pytest.raises(RuntimeError, match="gdr_step.cu:\\nbad kernel"):
        build.build()
    assert made(folder) == []
