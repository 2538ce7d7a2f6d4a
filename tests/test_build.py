"""What is compiled again, on the CPU, with a stand-in compiler that writes down its calls."""
import os
import time

import pytest

from nonlinear_rnn_solve_newton_b200 import build as b

NVCC = """#!/bin/sh
if [ "$1" = --version ]; then cat "{dir}/version"; exit 0; fi
for last; do :; done
echo "$@" >> "{dir}/calls"
echo made > "$last"
if [ -e "{dir}/edit" ]; then sleep 0.05; touch "$(cat "{dir}/edit")"; fi
"""


@pytest.fixture
def tree(tmp_path, monkeypatch):
    bin_ = tmp_path / "bin"
    bin_.mkdir()
    (tmp_path / "version").write_text("one\n")
    nvcc = bin_ / "nvcc"
    nvcc.write_text(NVCC.format(dir=tmp_path))
    nvcc.chmod(0o755)
    sources = []
    for name in ("x.cu", "y.cu"):
        (tmp_path / name).write_text('#include "both.cuh"\n')
        sources.append(str(tmp_path / name))
    (tmp_path / "both.cuh").write_text("\n")
    monkeypatch.setenv("PATH", f"{bin_}:{os.environ['PATH']}")
    for name, value in (("CSRC", str(tmp_path)), ("LIB", str(tmp_path / "lib.so")),
                        ("BUILD", str(tmp_path / "_build")), ("SOURCES", sources),
                        ("DEPS", [*sources, str(tmp_path / "both.cuh")])):
        monkeypatch.setattr(b, name, value)
    return tmp_path


def compiled(tree):
    """Sources compiled since the last look."""
    calls = tree / "calls"
    lines = calls.read_text().splitlines() if calls.exists() else []
    calls.write_text("")
    return sorted(os.path.basename(w) for line in lines if " -c " in line
                  for w in line.split() if w.endswith(".cu"))


def edit(path):
    time.sleep(0.05)
    os.utime(path)


def test_only_what_changed_is_compiled(tree):
    b.build()
    assert compiled(tree) == ["x.cu", "y.cu"] and not b.needs_build()
    edit(tree / "y.cu")
    assert b.needs_build()
    b.build()
    assert compiled(tree) == ["y.cu"]
    edit(tree / "both.cuh")
    b.build()
    assert compiled(tree) == ["x.cu", "y.cu"]


@pytest.mark.parametrize("what", ["flags", "compiler"])
def test_objects_of_other_settings_are_not_linked(tree, monkeypatch, what):
    b.build()
    compiled(tree)
    if what == "flags":
        flags = b._flags() + ["-DOTHER"]
        monkeypatch.setattr(b, "_flags", lambda: flags)
    else:
        (tree / "version").write_text("two\n")
    edit(tree / "y.cu")
    b.build()
    assert compiled(tree) == ["x.cu", "y.cu"]


def test_an_edit_during_the_build_is_compiled_again(tree):
    (tree / "edit").write_text(str(tree / "x.cu"))
    b.build()
    compiled(tree)
    (tree / "edit").unlink()
    assert b.needs_build()
    b.build()
    assert compiled(tree) == ["x.cu"] and not b.needs_build()


def test_each_process_writes_its_own_files(tree):
    b.build()
    outs = [line.split()[-1] for line in (tree / "calls").read_text().splitlines()]
    assert outs and all(f".{os.getpid()}." in os.path.basename(o) for o in outs)
    left = [*os.listdir(tree), *os.listdir(tree / "_build")]
    assert not any(n.endswith(".tmp") for n in left)
