"""The build's order and what it does without: libopq.so needs neither torch's nor Python's
C++ headers, only the extension over it does.  Compilers and linkers are stood in for."""
import os
import sys
import sysconfig

import pytest

from w4a16_linear_amd import build


@pytest.fixture
def steps(tmp_path, monkeypatch):
    """A build that records its steps, into tmp_path; an extension of an earlier build is there."""
    done = []
    for name in ("LIB", "CEILING_LIB", "EXT_LIB"):
        monkeypatch.setattr(build, name, str(tmp_path / os.path.basename(getattr(build, name))))
    monkeypatch.setattr(build, "OBJDIR", str(tmp_path / "obj"))
    monkeypatch.setattr(build, "_compile", lambda src, verbose: src + ".o")
    monkeypatch.setattr(build, "_compile_extension", lambda verbose: "ext.o")
    monkeypatch.setattr(build, "_link", lambda objs, lib, libs, verbose: done.append(os.path.basename(lib)))
    monkeypatch.setattr(build, "_link_extension", lambda obj, verbose: done.append("_attention.so"))
    (tmp_path / "_attention.so").write_text("old")
    return done


def test_everything(steps):
    assert build.build() == build.LIB
    assert steps == ["libopq.so", "libopq_ceiling.so", "_attention.so"] and os.path.exists(build.EXT_LIB)


@pytest.mark.parametrize("missing", ["Python.h", "torch", "torch headers"])
def test_libraries_without_the_extensions_needs(steps, missing, tmp_path, monkeypatch, capsys):
    if missing == "Python.h":
        monkeypatch.setattr(sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    elif missing == "torch":
        monkeypatch.setitem(sys.modules, "torch", None)      # an import of it raises ImportError
    else:
        import torch
        monkeypatch.setattr(torch, "__file__", str(tmp_path / "torch" / "__init__.py"))
    monkeypatch.setattr(build, "_compile_extension", lambda verbose: pytest.fail("compiled without its headers"))
    assert build.build() == build.LIB
    assert steps == ["libopq.so", "libopq_ceiling.so"] and not os.path.exists(build.EXT_LIB)
    assert "_attention.so" in capsys.readouterr().err


def test_a_failing_extension_leaves_the_libraries(steps, monkeypatch):
    def fail(verbose):
        raise RuntimeError("compile failed: attention_torch.cpp")

    monkeypatch.setattr(build, "_compile_extension", fail)
    with pytest.raises(RuntimeError, match="attention_torch"):
        build.build()
    assert steps == ["libopq.so", "libopq_ceiling.so"]
