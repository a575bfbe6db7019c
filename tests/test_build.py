"""The build: what is rebuilt when, and what a failure leaves."""

import os

import pytest

import tree_verification_verify_b200 as tv
from tree_verification_verify_b200 import build as b


@pytest.fixture
def tools(tmp_path, monkeypatch):
    """Compilers that note their runs and write their output file."""
    log = tmp_path / "log"
    script = '#!/bin/sh\necho $0 >> %s\nwhile [ "$1" != -o ]; do shift; done\n%secho x > $2\n%s'

    def tool(name, before="", after=""):
        path = tmp_path / name
        path.write_text(script % (log, before, after))
        path.chmod(0o755)
        return str(path)

    monkeypatch.setattr(b, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(b, "BINDING", str(tmp_path / "binding.so"))
    monkeypatch.setattr(b, "BINDING_FOR", str(tmp_path / "_build" / "for.txt"))
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


def test_a_binding_of_another_torch_is_not_loaded(monkeypatch):
    import torch
    b.build()
    monkeypatch.setattr(tv.paged, "_binding", None)
    monkeypatch.setattr(torch, "__version__", "99.1")
    with pytest.raises(tv.TVError, match="99.1.*build it again"):
        tv.paged.binding()
