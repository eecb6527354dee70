"""Which sources a build compiles again (no compiler needed: a stand-in writes the files)."""
from __future__ import annotations

import os
import shutil

import pytest

from cyclic_group_dft_b200 import build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A tree of two sources and a header, and the list of sources that were compiled."""
    csrc, obj = tmp_path / "csrc", tmp_path / "_build"
    csrc.mkdir()
    obj.mkdir()
    for name in ("a.cu", "b.cu", "h.cuh"):
        (csrc / name).write_text("")
        os.utime(csrc / name, (1, 1))
    monkeypatch.setattr(build, "ROOT", str(tmp_path))
    monkeypatch.setattr(build, "CSRC", str(csrc))
    monkeypatch.setattr(build, "OBJ", str(obj))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(build, "up_to_date", lambda: False)
    compiled = []

    def run(cmd, check):
        out = cmd[cmd.index("-o") + 1]
        if "-c" in cmd:
            src = next(c for c in cmd if c.endswith(".cu"))
            compiled.append((os.path.basename(src), [c for c in cmd if c.startswith("-D")]))
            with open(cmd[cmd.index("-MF") + 1], "w") as f:
                f.write(f"{out}: {src}" + (f" \\\n {csrc / 'h.cuh'}" if src.endswith("a.cu") else "") + "\n")
        with open(out, "w") as f:
            f.write("x")

    monkeypatch.setattr(build.subprocess, "run", run)

    def built(**kw):
        compiled.clear()
        build.build(**kw)
        return sorted(compiled)

    return tmp_path, built


def test_only_what_changed_is_compiled_again(tree):
    root, built = tree
    both = [("a.cu", []), ("b.cu", [])]
    assert built() == both
    assert built() == []
    later = os.path.getmtime(root / "_build" / "a.o") + 10
    os.utime(root / "csrc" / "h.cuh", (later, later))
    assert built() == [("a.cu", [])]                        # the one that includes it
    assert built(force=True) == both


def test_other_flags_compile_everything_again(tree):
    _, built = tree
    extra = [("a.cu", ["-DX"]), ("b.cu", ["-DX"])]
    built()
    assert built(extra=["-DX"]) == extra
    assert built() == [("a.cu", []), ("b.cu", [])]          # not the objects of the other flags
    assert built() == []


def test_a_copied_tree_does_not_use_the_objects_of_the_first(tree, monkeypatch, tmp_path_factory):
    root, built = tree
    built()
    copy = tmp_path_factory.mktemp("copy") / "tree"
    shutil.copytree(root, copy)
    for name, path in (("ROOT", copy), ("CSRC", copy / "csrc"), ("OBJ", copy / "_build")):
        monkeypatch.setattr(build, name, str(path))
    assert built() == [("a.cu", []), ("b.cu", [])]          # their dependency lists name the first tree's files


def test_a_failed_compile_leaves_no_record(tree, monkeypatch):
    root, built = tree

    def fail(cmd, check):
        raise build.subprocess.CalledProcessError(1, cmd)

    built()
    with monkeypatch.context() as m:
        m.setattr(build.subprocess, "run", fail)
        with pytest.raises(build.subprocess.CalledProcessError):
            build.build(extra=["-DX"])
    assert built() == []                                    # the first objects are whole, and still those of no flags
