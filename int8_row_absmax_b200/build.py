"""Build the BitLinear CUDA library in-tree for sm_100a, and the tensor binding of
its attention operators over it.

    python -m int8_row_absmax_b200.build        # -> int8_row_absmax_b200/libbitlinear.so, _binding.so

The library needs nvcc alone; the binding, which only PyTorch programs use, is left out
where PyTorch or the headers of PyTorch or Python are missing.  One nvcc invocation over one translation unit, and one of the host compiler.  No fast-math: the quantizers
need IEEE division and round-half-even, and -fmad=false keeps the dequant
epilogue from being contracted into an FMA.
"""
from __future__ import annotations

import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SRC = os.path.join(PKG, "csrc", "bitlinear_lib.cu")
OUT = os.path.join(PKG, "libbitlinear.so")
BINDING_SRC = os.path.join(PKG, "csrc", "torch_binding.cpp")
BINDING = os.path.join(PKG, "_binding.so")
ARCH = "-gencode=arch=compute_100a,code=sm_100a"


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    d = os.path.join(PKG, "csrc")
    return [os.path.join(d, f) for f in sorted(os.listdir(d)) if f.endswith((".cu", ".cuh"))] + \
        [os.path.join(ROOT, "include", "bitlinear.h")]


def binding_sources():
    return [BINDING_SRC, os.path.join(ROOT, "include", "bitlinear.h")]


def up_to_date(out: str = OUT, srcs=None) -> bool:
    if not os.path.exists(out):
        return False
    t = os.path.getmtime(out)
    return all(os.path.getmtime(s) <= t for s in (sources() if srcs is None else srcs))


def run(cmd, verbose: bool = False) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{os.path.basename(cmd[0])} failed:\n" + res.stdout + res.stderr)
    if verbose and (res.stdout or res.stderr):
        print(res.stdout + res.stderr)


def torch_root():
    """The folder of the installed PyTorch, or None (PyTorch itself is not imported)."""
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec is not None and spec.origin else None


def built_for() -> str:
    """What a binding has to be built for: the PyTorch and Python that run.  Part of the binding's bytes."""
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:                      # a PyTorch that was not installed as a package
        import torch
        version = torch.__version__
    return f"built for PyTorch {version}, Python {sys.version_info[0]}.{sys.version_info[1]};"


def binding_fits() -> bool:
    """Whether the binding is there and was built for the PyTorch and Python that run."""
    if not os.path.exists(BINDING):
        return False
    with open(BINDING, "rb") as f:
        return built_for().encode() in f.read()


def binding_lacks():
    """What the binding's build lacks here, in words, or None."""
    root = torch_root()
    if root is None:
        return "PyTorch is not installed"
    for header in (os.path.join(root, "include", "ATen", "ATen.h"),
                   os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        if not os.path.exists(header):
            return f"{header} is missing"
    return None


def build_binding(force: bool = False, verbose: bool = False) -> str:
    """The tensor binding, against the PyTorch that is installed."""
    if not force and up_to_date(BINDING, binding_sources()) and binding_fits():
        return BINDING
    import torch
    root = torch_root()
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include")]
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc_path()))), "include")
    run([shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-DTORCH_EXTENSION_NAME=_binding",
         f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DBL_BUILT_FOR="{built_for()}"',
         "-I", os.path.join(ROOT, "include"), "-isystem", cuda, "-isystem", sysconfig.get_paths()["include"],
         *(x for d in inc for x in ("-isystem", d)), BINDING_SRC, "-o", BINDING + ".tmp",
         "-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10", "-lc10_cuda", "-ldl"], verbose)
    os.replace(BINDING + ".tmp", BINDING)
    return BINDING


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    if force or not up_to_date():
        run([nvcc_path(), ARCH, "-O3", "-lineinfo", "-std=c++17", "-fmad=false",
             "-Xcompiler", "-fPIC", "-shared", "-Xptxas", "-warn-spills",
             "-I", os.path.join(ROOT, "include"), "-I", os.path.join(PKG, "csrc"),
             *extra, "-o", OUT + ".tmp", SRC], verbose)
        os.replace(OUT + ".tmp", OUT)
    lacks = binding_lacks()
    if lacks is not None:
        print(f"the tensor binding is not built: {lacks}", file=sys.stderr)
        return OUT
    try:
        build_binding(force, verbose)
    except RuntimeError as e:
        raise RuntimeError(f"{OUT} is built, its tensor binding is not: {e}") from e
    return OUT


if __name__ == "__main__":
    force = "--force" in sys.argv
    extra = ["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else []
    print(build(force=force or bool(extra), verbose=True, extra=extra))
