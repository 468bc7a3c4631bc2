"""What the build makes where torch, its headers or a compiler is missing (with stand-ins for the
compilers, which write what they are asked to)."""
import os
import sys

import pytest

WRITES = """#!/bin/sh
while [ $# -gt 0 ]; do [ "$1" = -o ] && : > "$2"; shift; done
"""


@pytest.fixture
def build(tmp_path, monkeypatch):
    from serving_step_sparse_gb300 import build as b
    compiler = tmp_path / "compiler"
    compiler.write_text(WRITES)
    compiler.chmod(0o755)
    monkeypatch.setattr(b, "NVCC", str(compiler))
    monkeypatch.setattr(b, "CXX", str(compiler))
    monkeypatch.setattr(b, "OUT_DIR", str(tmp_path / "out"))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "out" / "libula.so"))
    monkeypatch.setattr(b, "BINDING", str(tmp_path / "out" / "_rows.so"))
    return b


def test_builds_library_and_binding(build):
    assert not build.up_to_date()
    assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and os.path.exists(build.BINDING) and build.up_to_date()


def test_library_without_torch(build, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)             # as where it is not installed
    assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)
    assert build.up_to_date()
    monkeypatch.undo()


def test_binding_is_built_once_torch_is_there(build, monkeypatch):
    with monkeypatch.context() as m:
        m.setitem(sys.modules, "torch", None)
        build.build()
    assert not build.up_to_date()
    build.build()
    assert os.path.exists(build.BINDING) and build.up_to_date()


def test_library_stands_where_the_binding_fails(build, tmp_path, monkeypatch):
    monkeypatch.setattr(build, "CXX", "/bin/false")
    with pytest.raises(RuntimeError, match="rows_binding"):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)
    assert not build.up_to_date()


def test_no_library_where_a_source_fails(build, tmp_path, monkeypatch):
    monkeypatch.setattr(build, "NVCC", "/bin/false")
    with pytest.raises(RuntimeError, match="ula_kernels.cu"):
        build.build()
    assert not os.path.exists(build.LIB)
