"""In-tree build of libgqa_attn.so and libgqa_serve.so (nvcc, sm_100a only), and of the module that
binds the latter to Python."""
from __future__ import annotations

import glob
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libgqa_attn.so")
CSRC = os.path.join(HERE, "csrc")
SERVE_LIB = os.path.join(HERE, "libgqa_serve.so")
SERVE_CSRC = os.path.join(HERE, "csrc_serve")
SERVE_BIND = os.path.join(HERE, "_serve_bind.so")
SERVE_BIND_SRC = os.path.join(HERE, "bind", "serve_bind.cpp")
INCLUDE = os.path.join(ROOT, "include")

NVCC_FLAGS = [
    "-O3", "-std=c++17", "-lineinfo",
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-shared", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "--expt-relaxed-constexpr",
]


def sources():
    return _sources(CSRC)


def _sources(folder):
    return sorted(glob.glob(os.path.join(folder, "*.cu")) + glob.glob(os.path.join(folder, "*.cpp")))


def _headers(folder):
    return [f for e in ("*.h", "*.cuh") for f in glob.glob(os.path.join(folder, e))]


def _stale() -> bool:
    return _older(LIB, sources() + _headers(CSRC))


def serve_stale() -> bool:
    # the serving kernels share the forward's device headers
    return _older(SERVE_LIB, _sources(SERVE_CSRC) + _headers(SERVE_CSRC) + _headers(CSRC))


def bind_stale() -> bool:
    return _older(SERVE_BIND, [SERVE_BIND_SRC]) or _bind_made_for() != _bind_abi()


def _bind_abi() -> str:
    """What the binding is compiled against."""
    import torch
    return f"{sys.implementation.cache_tag} torch {torch.__version__}"


def _bind_made_for():
    # written beside the module once it is built
    try:
        with open(SERVE_BIND + ".stamp") as f:
            return f.read()
    except OSError:
        return None


def _older(lib, deps) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(d) > t for d in deps + _headers(INCLUDE))


def _compile(lib, folders, files, verbose):
    cmd = ["nvcc", *NVCC_FLAGS, "-I", INCLUDE]
    for f in folders:
        cmd += ["-I", f]
    if verbose:
        cmd += ["-Xptxas", "-v"]
    subprocess.run(cmd + ["-o", lib, *files, "-ldl"], check=True)
    return lib


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the forward's library if any source is newer than it (nvcc alone is needed); return
    its path."""
    if not force and not _stale():
        return LIB
    return _compile(LIB, [CSRC], sources(), verbose)


def build_serve(force: bool = False, verbose: bool = False) -> str:
    if not force and not serve_stale():
        return SERVE_LIB
    return _compile(SERVE_LIB, [SERVE_CSRC, CSRC], _sources(SERVE_CSRC), verbose)


def build_bind(force: bool = False) -> str:
    """The binding module, against this interpreter and torch; it finds libgqa_serve.so beside it."""
    if not force and not bind_stale():
        return SERVE_BIND
    import sysconfig

    import torch
    from torch.utils import cpp_extension

    paths = [INCLUDE, sysconfig.get_paths()["include"], *cpp_extension.include_paths("cuda")]
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    cmd = ["g++", "-O2", "-std=c++20", "-fPIC", "-shared", "-fvisibility=hidden", "-w",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}"]
    for p in paths:
        cmd += ["-isystem", p]
    cmd += [SERVE_BIND_SRC, "-o", SERVE_BIND, "-L", HERE, "-l:libgqa_serve.so", "-Wl,-rpath,$ORIGIN",
            "-L", libs, "-lc10", "-lc10_cuda", "-ltorch", "-ltorch_cpu", "-ltorch_python"]
    if os.path.exists(SERVE_BIND + ".stamp"):
        os.remove(SERVE_BIND + ".stamp")
    subprocess.run(cmd, check=True)
    with open(SERVE_BIND + ".stamp", "w") as f:
        f.write(_bind_abi())
    return SERVE_BIND


def build_all(force: bool = False, verbose: bool = False) -> None:
    """The forward's library, the serving library and, with torch, the latter's binding."""
    build(force, verbose)
    build_serve(force, verbose)
    build_bind(force)


if __name__ == "__main__":
    build_all(force=True, verbose=True)
