"""When the library is compiled again (CPU; the compiler is a script that writes its output file)."""
import os

import pytest

from gated_delta_rule_91_b200 import _build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    csrc = tmp_path / "csrc"
    csrc.mkdir()
    (csrc / "a.cu").write_text('#include "shared.cuh"\n')
    (csrc / "b.cu").write_text('#include "shared.cuh"\n#include "own.cuh"\n')
    (csrc / "shared.cuh").write_text("\n")
    (csrc / "own.cuh").write_text("\n")
    log = tmp_path / "log"
    nvcc = tmp_path / "nvcc"
    nvcc.write_text('#!/bin/sh\necho "$@" >> %s\nwhile [ $# -gt 0 ]; do if [ "$1" = -o ]; then touch "$2"; fi; shift; done\n' % log)
    nvcc.chmod(0o755)
    monkeypatch.setattr(_build, "CSRC", str(csrc))
    monkeypatch.setattr(_build, "ROOT", str(tmp_path))
    monkeypatch.setattr(_build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(_build, "UNITS", ("a", "b"))
    monkeypatch.setenv("NVCC", str(nvcc))

    class Tree:
        path = csrc

        def calls(self):
            n = len(log.read_text().splitlines()) if log.exists() else 0
            if log.exists():
                log.unlink()
            return n

        def age(self, name, seconds):
            f = tmp_path / name if (tmp_path / name).exists() else csrc / name
            t = os.path.getmtime(f) + seconds
            os.utime(f, (t, t))

    return Tree()


def test_units_that_changed_are_compiled(tree):
    _build.build()
    assert tree.calls() == 3  # two units and the link
    for f in ("a.cu", "b.cu", "shared.cuh", "own.cuh"):
        tree.age(f, -100)
    _build.build()
    assert tree.calls() == 0
    tree.age("own.cuh", 300)
    _build.build()
    assert tree.calls() == 2  # one unit and the link


def test_a_library_newer_than_its_sources_needs_no_objects(tree):
    """A tree with the built library alone, where no compiler may be."""
    _build.build()
    tree.calls()
    for f in ("a.cu", "b.cu", "shared.cuh", "own.cuh"):
        tree.age(f, -100)
    os.remove(tree.path / "a.o")
    os.remove(tree.path / "b.o")
    assert _build.build() == _build.LIB
    assert tree.calls() == 0
    _build.build(force=True)
    assert tree.calls() == 3
