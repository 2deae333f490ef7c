"""What the build does where the tensor front end cannot be built, and when the library comes into a process."""
import os
import subprocess
import sys

import pytest

from gate_cores_b200 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Spec:
    def __init__(self, where):
        self.submodule_search_locations = [str(where)]


def no_compiler(*a, **k):
    raise AssertionError("the compiler was called")


@pytest.fixture
def front(monkeypatch, tmp_path):
    """An extension built for something else."""
    old = tmp_path / "_front.so"
    old.write_text("old")
    monkeypatch.setattr(build, "FRONT", str(old))
    return old


def test_a_pytorch_without_cuda(monkeypatch, tmp_path, capsys, front):
    # the C library is complete without the front end: nothing is compiled, nothing raised, and why is said
    (tmp_path / "lib").mkdir()
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: Spec(tmp_path))
    monkeypatch.setattr(build.subprocess, "check_call", no_compiler)
    build._build_front(True)
    assert "without CUDA" in capsys.readouterr().err and not front.exists()


def test_no_cxx_compiler(monkeypatch, capsys, front):
    which = build.shutil.which
    monkeypatch.setattr(build.shutil, "which", lambda name, *a, **k: None if name == "g++" else which(name, *a, **k))
    monkeypatch.setattr(build.subprocess, "check_call", no_compiler)
    build._build_front(True)
    assert "no g++" in capsys.readouterr().err and not front.exists()


def test_a_front_end_that_is_up_to_date_needs_no_compiler(monkeypatch):
    build.build()
    monkeypatch.setattr(build.shutil, "which", lambda *a, **k: None)
    monkeypatch.setattr(build.subprocess, "check_call", no_compiler)
    build._build_front(False)
    assert os.path.exists(build.FRONT)


def test_a_compiler_that_fails_is_an_error(monkeypatch, front):
    def fails(cmd, *a, **k):
        raise subprocess.CalledProcessError(1, cmd)

    monkeypatch.setattr(build.subprocess, "check_call", fails)
    with pytest.raises(subprocess.CalledProcessError):
        build._build_front(True)


def test_the_library_comes_with_the_first_call():
    # a program that imports the package, builds, and calls must run what it has built: nothing is loaded before a call
    code = """
import torch
import gate_cores_b200
from gate_cores_b200 import cores
loaded = lambda: [l.split()[-1] for l in open("/proc/self/maps") if "gate_cores_b200" in l and ".so" in l]
assert not loaded(), loaded()
try:
    cores.layer_norm(torch.zeros(4, 64))
except ValueError:
    pass
assert any("libmuse_cores" in l for l in loaded()) and any("_front" in l for l in loaded())
"""
    build.build()
    subprocess.run([sys.executable, "-c", code], check=True, cwd=ROOT, timeout=300)
