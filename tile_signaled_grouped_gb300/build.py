"""Build the in-tree shared library libmoe_tsg.so for sm_103a with nvcc, and its torch
binding _torch_ops.so with the host compiler.

Each translation unit compiles in parallel into _build/, then one nvcc link
produces tile_signaled_grouped_gb300/libmoe_tsg.so (CUDA runtime linked
statically, so the library needs only the driver at run time) and one host link the
binding, which loads that library from its own folder. Where PyTorch or the headers that
the binding needs are not installed, the library is built alone.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmoe_tsg.so")
BINDING = os.path.join(PKG, "_torch_ops.so")
SOURCES = ["api.cu", "plan.cu", "ffn.cu", "ffn_pair.cu", "consumer.cu", "route_scale.cu", "gate.cu",
           "plan_noalloc.cu", "gate_rows.cu", "router.cu", "norm.cu",
           "linear.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _flags(extra=()):
    return ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
                   "-I", os.path.join(ROOT, "include"), *extra]


def _compile(src: str, verbose: bool, extra) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc(), *_flags(extra), "-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        sys.stderr.write(r.stdout + r.stderr)
    return obj


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def _torch():
    """PyTorch's folder, or None where it is not installed."""
    spec = importlib.util.find_spec("torch")
    return None if spec is None else os.path.dirname(spec.origin)


def binding_lacks():
    """What the torch binding's build lacks here, in words, or None."""
    if _torch() is None:
        return "PyTorch is not installed"
    for f in (os.path.join(_torch(), "include", "torch", "extension.h"),
              os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        if not os.path.exists(f):
            return f"{f} is missing"
    return None if shutil.which(_cxx()) else f"no host compiler ({_cxx()})"


def _cxx() -> str:
    return os.environ.get("CXX", "g++")


def _built_for() -> str:
    """What a binding fits: the Python and the PyTorch it was compiled against."""
    with open(os.path.join(_torch(), "version.py")) as f:
        return f"{sysconfig.get_config_var('SOABI')}\n{_torch()}\n{f.read()}"


def _binding_fits() -> bool:
    try:
        with open(os.path.join(BUILD, "torch_ops.for")) as f:
            return f.read() == _built_for()
    except OSError:
        return False


def _compile_binding() -> str:
    obj = os.path.join(BUILD, "torch_ops.o")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    inc = [os.path.join(_torch(), "include"),
           os.path.join(_torch(), "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    _run([_cxx(), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
          *[f for i in inc for f in ("-isystem", i)], "-DTORCH_EXTENSION_NAME=_torch_ops", "-c",
          os.path.join(CSRC, "torch_ops.cpp"), "-o", obj], "the torch binding's compilation")
    return obj


def _stale() -> bool:
    made = [LIB] if binding_lacks() else [LIB, BINDING]
    if not all(map(os.path.exists, made)) or (BINDING in made and not _binding_fits()):
        return True
    t = min(map(os.path.getmtime, made))
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    deps.append(os.path.join(ROOT, "include", "moe_tsg.h"))
    deps.append(os.path.abspath(__file__))
    return any(os.path.getmtime(p) > t for p in deps)


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    """Compile and link; returns the library path. Rebuilds only when sources changed, or what
    the binding was compiled against."""
    if not force and not _stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = None if binding_lacks() else ex.submit(_compile_binding)
        objs = list(ex.map(lambda s: _compile(s, verbose, extra), SOURCES))
    tmp = LIB + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    _run(cmd, "nvcc link")
    os.replace(tmp, LIB)
    if binding is None:
        return LIB
    tmp = BINDING + ".tmp"
    _run([_cxx(), "-shared", "-o", tmp, binding.result(), "-L" + PKG,
          "-l:libmoe_tsg.so", "-L" + os.path.join(_torch(), "lib"), "-lc10", "-lc10_cuda",
          "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN"], "the torch binding's link")
    os.replace(tmp, BINDING)
    with open(os.path.join(BUILD, "torch_ops.for"), "w") as f:
        f.write(_built_for())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
