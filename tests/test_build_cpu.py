"""The library takes hipcc alone; the binding's module is built where it can be."""
import os
import subprocess
import sys

import pytest

from lora_moe_amd import build

TINY = 'extern "C" int answer() { return 42; }\n'


@pytest.fixture
def tiny(tmp_path, monkeypatch):
    """A library of one function, built into a folder of its own."""
    (tmp_path / "tiny.hip").write_text(TINY)
    for n in ("OBJ", "SO", "OPERANDS"):
        monkeypatch.setattr(build, n, str(tmp_path / n.lower()))
    monkeypatch.setattr(build, "sources", lambda: [str(tmp_path / "tiny.hip")])
    return tmp_path


def answer(path):
    # (in a process of its own: this one may hold torch's HIP runtime)
    code = f"import ctypes; raise SystemExit(ctypes.CDLL({path!r}).answer())"
    return subprocess.run([sys.executable, "-c", code]).returncode


def test_both_are_built(tiny):
    assert build.build() == build.SO and answer(build.SO) == 42 and os.path.exists(build.OPERANDS)


@pytest.mark.parametrize("missing", ["torch", "compiler", "headers"])
def test_the_library_does_not_need_the_module(tiny, monkeypatch, missing):
    open(build.OPERANDS, "w").close()  # of an earlier build
    if missing == "torch":
        monkeypatch.setitem(sys.modules, "torch", None)
    elif missing == "compiler":
        run = subprocess.run
        monkeypatch.setattr(build.subprocess, "run", lambda a, **k: run(["false"] if "operands.c" in " ".join(a) else a, **k))
    else:
        monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": str(tiny)})
    with pytest.warns(UserWarning, match="_operands is not"):
        assert build.build() == build.SO
    assert answer(build.SO) == 42 and not os.path.exists(build.OPERANDS)
