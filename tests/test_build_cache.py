"""Which objects a build takes over: those of the same sources, flags and
compiler, and no others (CPU, with a stand-in for the compiler)."""
import os
import stat

import pytest

from selective_state_space_51_b200 import build as B

NVCC = """#!/bin/sh
if [ "$1" = --version ]; then cat "%(at)s/version"; exit 0; fi
echo "$@" >> "%(at)s/calls"
for last; do :; done
out=""; prev=""
for a in "$@"; do [ "$prev" = -o ] && out="$a"; prev="$a"; done
echo "$@" > "$out"
"""


@pytest.fixture
def tree(tmp_path, monkeypatch):
    csrc, inc = tmp_path / "csrc", tmp_path / "include"
    csrc.mkdir()
    inc.mkdir()
    (csrc / "a.cu").write_text('#include "h.cuh"\n')
    (csrc / "b.cu").write_text("int b;\n")
    (csrc / "h.cuh").write_text("int h;\n")
    (tmp_path / "version").write_text("release 1\n")
    nvcc = tmp_path / "nvcc"
    nvcc.write_text(NVCC % dict(at=tmp_path))
    nvcc.chmod(nvcc.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setattr(B, "_nvcc", lambda: str(nvcc))
    monkeypatch.setattr(B, "CSRC", str(csrc))
    monkeypatch.setattr(B, "INCLUDE", str(inc))
    monkeypatch.setattr(B, "OBJECTS", str(tmp_path / "_build"))
    monkeypatch.setattr(B, "LIB", str(tmp_path / "lib.so"))
    old = 1_000_000_000
    for p in (csrc / "a.cu", csrc / "b.cu", csrc / "h.cuh"):
        os.utime(p, (old, old))
    return tmp_path


def calls(tree, **kw):
    """What a build compiles (and links), by the sources' names."""
    log = tree / "calls"
    if log.exists():
        log.unlink()
    B.build(**kw)
    if not log.exists():
        return []
    return sorted(os.path.basename(line.split()[-1]) if " -c " in line
                  else "link" for line in log.read_text().splitlines())


ALL = ["a.cu", "b.cu", "link"]


def test_nothing_changed(tree):
    assert calls(tree) == ALL
    assert calls(tree) == []
    assert calls(tree, force=True) == ALL


def test_a_header_rebuilds_what_includes_it(tree):
    calls(tree)
    far = os.path.getmtime(B.LIB) + 100
    os.utime(tree / "csrc" / "h.cuh", (far, far))
    assert calls(tree) == ["a.cu", "link"]


def test_other_flags_share_no_objects(tree):
    calls(tree)
    assert calls(tree, extra=("-DX",)) == ALL
    assert calls(tree, extra=("-DX",)) == []
    assert calls(tree) == ALL
    for o in ("a.o", "b.o"):
        assert "-DX" not in (tree / "_build" / o).read_text()


def test_other_flags_after_an_edit_share_no_objects(tree):
    calls(tree, extra=("-DX",))
    far = os.path.getmtime(B.LIB) + 100
    os.utime(tree / "csrc" / "h.cuh", (far, far))
    assert calls(tree) == ALL


def test_changed_flags_or_compiler_rebuild(tree, monkeypatch):
    calls(tree)
    monkeypatch.setattr(B, "NVCC_FLAGS", B.NVCC_FLAGS + ["-Xptxas", "-v"])
    assert calls(tree) == ALL
    (tree / "version").write_text("release 2\n")
    assert calls(tree) == ALL
    assert calls(tree) == []


def test_a_broken_build_is_not_taken_for_a_finished_one(tree):
    calls(tree)
    os.remove(tree / "_build" / "lib.so.key")
    assert calls(tree) == ["link"]


def test_without_a_compiler_the_library_is_taken_by_its_date(tree,
                                                             monkeypatch):
    calls(tree)

    def none():
        raise RuntimeError("nvcc not found")

    monkeypatch.setattr(B, "_nvcc", none)
    assert B.build() == B.LIB
    far = os.path.getmtime(B.LIB) + 100
    os.utime(tree / "csrc" / "h.cuh", (far, far))
    with pytest.raises(RuntimeError):
        B.build()
