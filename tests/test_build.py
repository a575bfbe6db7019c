"""The build: what is rebuilt when, and what a failure leaves."""

import os
import subprocess

import pytest

import tree_verification_verify_b200 as tv
from tree_verification_verify_b200 import build as b


@pytest.fixture
def tools(tmp_path, monkeypatch):
    """Compilers that note their runs and write their arguments to their output file."""
    log = tmp_path / "log"
    script = '#!/bin/sh\necho $0 >> %s\nall="$*"\nwhile [ "$1" != -o ]; do shift; done\n%secho "$all" > $2\n%s'

    def tool(name, before="", after=""):
        path = tmp_path / name
        path.write_text(script % (log, before, after))
        path.chmod(0o755)
        return str(path)

    monkeypatch.setattr(b, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(b, "BINDING", str(tmp_path / "binding.so"))
    monkeypatch.setenv("NVCC", tool("nvcc"))
    monkeypatch.setenv("CXX", tool("cxx"))

    def runs():
        names = [os.path.basename(x) for x in log.read_text().split()] if log.exists() else []
        log.write_text("")
        return sorted(names)

    tool.runs = runs
    return tool


def test_only_what_is_out_of_date_is_built(tools):
    b.build()
    assert tools.runs() == ["cxx", "nvcc"]
    b.build()
    assert tools.runs() == []
    b.build(force=True)
    assert tools.runs() == ["cxx", "nvcc"]


def test_another_torch_rebuilds_the_binding(tools, monkeypatch):
    import torch
    b.build()
    tools.runs()
    monkeypatch.setattr(torch, "__version__", "99.1")
    b.build()
    assert tools.runs() == ["cxx"]
    b.build()
    assert tools.runs() == []


def test_the_binding_says_what_it_was_built_against():
    b.build()
    assert b.binding_built_against() == b.binding_against()


def test_a_binding_of_another_torch_is_not_loaded(monkeypatch):
    import torch
    b.build()
    monkeypatch.setattr(tv.paged, "_binding", None)
    monkeypatch.setattr(torch, "__version__", "99.1")
    with pytest.raises(tv.TVError, match="99.1.*build it again"):
        tv.paged.binding()


def test_the_library_stands_by_itself(tools, monkeypatch):
    """Without a C++ compiler, or with one that fails, the library is built and the user warned."""
    for cxx in (tools("cxx_fails", before="exit 1\n"), "/nonexistent/cxx"):
        monkeypatch.setenv("CXX", cxx)
        with pytest.warns(UserWarning, match="binding of the paged calls was not built"):
            assert b.build(force=True) == b.LIB
        assert os.path.exists(b.LIB) and not os.path.exists(b.BINDING)
        os.remove(b.LIB)
    monkeypatch.setenv("CXX", tools("cxx"))
    tools.runs()
    b.build()
    assert tools.runs() == ["cxx", "nvcc"] and os.path.exists(b.BINDING)


def test_a_failed_library_leaves_nothing_running(tools, monkeypatch, tmp_path):
    """The error comes when the other compiler has ended, and its output is in place."""
    monkeypatch.setenv("NVCC", tools("nvcc_fails", before="exit 1\n"))
    monkeypatch.setenv("CXX", tools("cxx_slow", before="sleep 1\n", after=f"echo end > {tmp_path}/ended"))
    with pytest.raises(subprocess.CalledProcessError):
        b.build()
    assert (tmp_path / "ended").exists() and os.path.exists(b.BINDING) and not os.path.exists(b.LIB)
