"""What build.py builds, with the compilers replaced by a recorder: libqmoe.so does not depend on
PyTorch, and the binding follows the PyTorch and Python that it is for."""

import os
import subprocess

import pytest

from quantized_moe_grouped_route_gb300 import build


@pytest.fixture
def runs(tmp_path, monkeypatch):
    """The outputs of the commands that a build ran; a command's output is an empty file."""
    made = []

    def run(cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        open(out, "w").close()
        made.append(os.path.basename(out).replace(".tmp", ""))
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build.subprocess, "run", run)
    for name, path in (("BUILD", "b"), ("LIBDIR", "l"), ("LIB", "l/libqmoe.so"),
                       ("BINDING", "l/qmoe_torch.so"), ("BINDING_FOR", "b/qmoe_torch.for")):
        monkeypatch.setattr(build, name, str(tmp_path / path))
    monkeypatch.setattr(build, "_torch_version", lambda: "one")
    return made


OBJECTS = {os.path.splitext(s)[0] + ".o" for s in build.SOURCES}
ALL = OBJECTS | {"libqmoe.so", "binding.o", "qmoe_torch.so"}


def test_builds_what_is_stale(runs, monkeypatch):
    build.build()
    assert set(runs) == ALL
    runs.clear()
    build.build()
    assert runs == []
    build.build(force=True)
    assert set(runs) == ALL
    runs.clear()
    os.remove(build.LIB)
    build.build()
    assert set(runs) == OBJECTS | {"libqmoe.so"}


def test_another_torch_gets_a_binding_of_its_own(runs, monkeypatch):
    build.build()
    runs.clear()
    monkeypatch.setattr(build, "_torch_version", lambda: "two")
    build.build()
    assert runs == ["binding.o", "qmoe_torch.so"]
    runs.clear()
    build.build()
    assert runs == []


def test_without_a_torch_that_has_cuda(runs, monkeypatch):
    monkeypatch.setattr(build, "_torch_version", lambda: None)
    build.build()
    assert set(runs) == OBJECTS | {"libqmoe.so"}
    assert not os.path.exists(build.BINDING)
    runs.clear()
    build.build()
    assert runs == []


def test_a_binding_that_fails_leaves_the_library(runs, monkeypatch):
    def fail():
        raise RuntimeError("no such header")
    monkeypatch.setattr(build, "_compile_binding", fail)
    with pytest.raises(RuntimeError, match="no such header"):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)


def test_versions_name_torch_and_python():
    import sys

    import torch
    version = build._torch_version()
    if torch.version.cuda:
        assert torch.__version__ in version and sys.version.split()[0] in version
    else:
        assert version is None
