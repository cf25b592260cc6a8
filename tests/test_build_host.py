"""The in-tree builds on the host: what each needs, what a failed one does, and when one is stale.
Nothing is compiled: the compilers are replaced by a record of their commands."""
import importlib.util
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

_WITHOUT_TORCH = r"""
import sys
sys.modules["torch"] = None  # import torch raises ImportError
import gqa_exact_attention_b200 as G
from gqa_exact_attention_b200 import _build
built = []
_build.subprocess.run = lambda cmd, **kw: built.append(cmd[cmd.index("-o") + 1])
_build._older = lambda lib, deps: True
_build.build()
assert built == [_build.LIB], built
G._have_nvcc = lambda: True
G.load()
assert built == [_build.LIB] * 2, built
print("built")
"""


def test_the_forward_builds_and_loads_without_torch():
    r = subprocess.run([sys.executable, "-c", _WITHOUT_TORCH], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.split() == ["built"], r.stderr


@pytest.fixture
def build(monkeypatch):
    """A fresh copy of the build module that only records its commands."""
    spec = importlib.util.spec_from_file_location("gqa_build_copy", os.path.join(ROOT, "gqa_exact_attention_b200", "_build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    mod.commands = []
    monkeypatch.setattr(mod, "subprocess", type("Record", (), {"run": staticmethod(lambda cmd, **kw: mod.commands.append(cmd))}))
    return mod


def test_build_all_builds_the_binding_after_its_library(build):
    build.build_all(force=True)
    assert [c[c.index("-o") + 1] for c in build.commands] == [build.LIB, build.SERVE_LIB, build.SERVE_BIND]


_FAILING = r"""
import subprocess, sys
import gqa_exact_attention_b200 as G
from gqa_exact_attention_b200 import _build, serving
G._have_nvcc = serving._have_nvcc = lambda: True
def run(cmd, **kw):
    raise subprocess.CalledProcessError(1, cmd)
_build.subprocess = type("S", (), {"run": staticmethod(run)})
which, stale = sys.argv[1:]
real = _build._older
_build._older = lambda lib, deps: lib.endswith(stale) or real(lib, deps)
try:
    {"forward": G.load, "serving": G.load_serve, "binding": serving._load_bind}[which]()
    print("loaded")
except RuntimeError as e:
    print("refused", stale in str(e))
"""


@pytest.mark.parametrize("which,stale,want", [
    ("forward", "libgqa_attn.so", "refused True"), ("serving", "libgqa_serve.so", "refused True"),
    ("binding", "_serve_bind.so", "refused True"), ("binding", "libgqa_serve.so", "refused True"),
    ("forward", "_serve_bind.so", "loaded"), ("serving", "_serve_bind.so", "loaded")])
def test_a_failed_build_does_not_hide_behind_an_old_library(which, stale, want):
    pytest.importorskip("torch")
    r = subprocess.run([sys.executable, "-c", _FAILING, which, stale], cwd=ROOT, capture_output=True, text=True)
    assert r.stdout.strip() == want, r.stdout + r.stderr


def test_a_binding_built_for_another_torch_is_stale(build, tmp_path, monkeypatch):
    torch = pytest.importorskip("torch")
    so = tmp_path / "_serve_bind.so"
    monkeypatch.setattr(build, "SERVE_BIND", str(so))

    def run(cmd, **kw):
        so.write_bytes(b"")
    monkeypatch.setattr(build.subprocess, "run", staticmethod(run))
    assert build.bind_stale()
    build.build_bind()
    assert not build.bind_stale()
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    assert build.bind_stale()
    build.build_bind()
    assert not build.bind_stale()
    monkeypatch.setattr(build.sys.implementation, "cache_tag", "cpython-300")
    assert build.bind_stale()


def test_a_failed_build_of_the_binding_leaves_it_stale(build, tmp_path, monkeypatch):
    pytest.importorskip("torch")
    so = tmp_path / "_serve_bind.so"
    monkeypatch.setattr(build, "SERVE_BIND", str(so))

    def run(cmd, **kw):
        so.write_bytes(b"")  # (some of it)
        raise OSError("no space")
    monkeypatch.setattr(build.subprocess, "run", staticmethod(run))
    with pytest.raises(OSError):
        build.build_bind()
    assert build.bind_stale()
