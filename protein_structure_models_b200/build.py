"""Build libfipa.so (the C-ABI library) in-tree with nvcc for sm_100a, and
_native.so (the compiled calls of the sequence operators from Python) with g++.

Usage: python -m protein_structure_models_b200.build
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libfipa.so")
NATIVE = os.path.join(PKG, "_native.so")
NATIVE_SOURCE = os.path.join(CSRC, "binding.cpp")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC,-fvisibility=hidden",
    "--expt-relaxed-constexpr",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale(target, deps) -> bool:
    return not os.path.exists(target) or any(os.path.getmtime(d) > os.path.getmtime(target) for d in deps)


def _headers():
    return glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))


def needs_build() -> bool:
    return _stale(LIB, sources() + _headers())


def _run(cmd) -> str:
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed:\n" + " ".join(cmd) + "\n" + res.stdout + res.stderr)
    return res.stdout + res.stderr


def built_for() -> str:
    """What the Python calls are compiled against; the module carries it as its documentation."""
    import sysconfig

    import torch
    return f"Calls of the sequence operators for {sysconfig.get_config_var('SOABI')}, PyTorch {torch.__version__}, " \
        f"C++ ABI {int(torch._C._GLIBCXX_USE_CXX11_ABI)}."


def native_needs_build() -> bool:
    """Older than its sources, or made for another Python or PyTorch, whose interfaces it would not fit (found without loading it)."""
    if _stale(NATIVE, [NATIVE_SOURCE, os.path.join(INCLUDE, "fipa.h")]):
        return True
    with open(NATIVE, "rb") as f:
        return built_for().encode() + b"\0" not in f.read()


def build_native(force: bool = False) -> str:
    """Compile the Python calls against the headers of Python and PyTorch; returns the module's path."""
    import sysconfig

    import torch
    if not force and not native_needs_build():
        return NATIVE
    home = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    inc = [INCLUDE, os.path.join(home, "include"), os.path.join(home, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    _run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DFIPA_BUILT_FOR="{built_for()}"', *[f"-I{d}" for d in inc], NATIVE_SOURCE,
          "-o", NATIVE + ".tmp", "-L" + os.path.join(home, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"])
    os.replace(NATIVE + ".tmp", NATIVE)
    return NATIVE


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every CUDA source into one shared library (the sources side by side),
    and the Python calls; returns the library's path."""
    if force or needs_build():
        nvcc = os.environ.get("NVCC", "nvcc")
        flags = [*NVCC_FLAGS, *(["-Xptxas=-v"] if verbose else []), "-I", INCLUDE, "-I", CSRC]
        with tempfile.TemporaryDirectory() as tmp, ThreadPoolExecutor(max(1, os.cpu_count() or 1)) as pool:
            objects = [os.path.join(tmp, os.path.basename(s)[:-3] + ".o") for s in sources()]
            for log in pool.map(lambda so: _run([nvcc, *flags, "-c", so[0], "-o", so[1]]), zip(sources(), objects)):
                if verbose:
                    sys.stderr.write(log)
            _run([nvcc, *NVCC_FLAGS[:2], "-shared", "-Xcompiler", "-fPIC", *objects, "-o", LIB + ".tmp"])
        os.replace(LIB + ".tmp", LIB)
    build_native(force)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
