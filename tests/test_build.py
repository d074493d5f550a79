"""What the build needs: the library hipcc alone; the binding for torch, where torch is, also a host compiler.  The
compilers are scripts here that write the file they are asked for."""
import os
import stat

import pytest

from gated_delta_rule_scan_amd import build as b


@pytest.fixture
def tree(tmp_path, monkeypatch):
    def compiler(name, status=0):
        p = tmp_path / name
        p.write_text('#!/bin/sh\nif [ %d != 0 ]; then echo broken; exit %d; fi\n'
                     'while [ $# != 0 ]; do if [ "$1" = -o ]; then echo %s > "$2"; fi; shift; done\n' % (status, status, name))
        p.chmod(p.stat().st_mode | stat.S_IXUSR)
        return str(p)

    monkeypatch.setenv("HIPCC", compiler("hipcc"))
    monkeypatch.setenv("CXX", compiler("cxx"))
    monkeypatch.setattr(b, "BUILD_DIR", str(tmp_path / "objects"))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(b, "BINDING", str(tmp_path / "binding.so"))
    return compiler


def _hide(monkeypatch, module):
    real = b.importlib.util.find_spec
    monkeypatch.setattr(b.importlib.util, "find_spec", lambda name, *a: None if name == module else real(name, *a))


def test_both_are_built(tree):
    assert b.build() == b.LIB
    assert open(b.LIB).read() == "hipcc\n" and open(b.BINDING).read() == "cxx\n"


def test_without_torch_the_library_is_built(tree, monkeypatch, capsys):
    _hide(monkeypatch, "torch")
    assert b.build() == b.LIB and os.path.exists(b.LIB)
    assert not os.path.exists(b.BINDING) and "binding" in capsys.readouterr().err


def test_without_a_host_compiler_the_library_is_built(tree, monkeypatch, tmp_path, capsys):
    monkeypatch.setenv("CXX", str(tmp_path / "no such compiler"))
    assert b.build() == b.LIB and os.path.exists(b.LIB)
    assert not os.path.exists(b.BINDING) and "binding" in capsys.readouterr().err


def test_without_python_headers_the_library_is_built(tree, monkeypatch, tmp_path, capsys):
    monkeypatch.setattr(b.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    assert b.build() == b.LIB and os.path.exists(b.LIB)
    assert not os.path.exists(b.BINDING) and "binding" in capsys.readouterr().err


def test_a_binding_that_fails_leaves_the_library(tree, monkeypatch):
    monkeypatch.setenv("CXX", tree("broken", 1))
    open(b.BINDING, "w").write("of the library before")
    with pytest.raises(RuntimeError, match="gdn_binding.cpp"):
        b.build()
    assert os.path.exists(b.LIB) and not os.path.exists(b.BINDING)


def test_a_source_that_fails_replaces_nothing(tree, monkeypatch):
    monkeypatch.setenv("HIPCC", tree("broken", 1))
    with pytest.raises(RuntimeError):
        b.build()
    assert not os.path.exists(b.LIB) and not os.path.exists(b.BINDING)
