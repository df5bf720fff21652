"""Build the sm_100a shared library in-tree with nvcc.

``libfp4moe.so`` is the product library; ``libfp4moe_checked.so`` is the same
sources with the device bounds checks compiled in (-DMOE_DEBUG_CHECKS): every
index a kernel reads from device data is checked before use and a bad one is
reported through the layer's error word instead of faulting.  The package
loads the checked library when FP4MOE_CHECKED=1 is set in the environment.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import runpy
import shutil
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
SO = os.path.join(HERE, "libfp4moe.so")
SO_CHECKED = os.path.join(HERE, "libfp4moe_checked.so")
SO_BINDING = os.path.join(HERE, "_ops.so")
CUDA_ROOTS = (os.environ.get("CUDA_HOME"), os.environ.get("CUDA_PATH"), "/usr/local/cuda")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))


def up_to_date(so: str = SO) -> bool:
    if not os.path.exists(so):
        return False
    t = os.path.getmtime(so)
    return all(os.path.getmtime(d) <= t for d in _deps())


def nvcc_cmd(out: str, extra=()):
    return (["nvcc", "-O3", "-std=c++17", *ARCH, "-lineinfo", "-Xcompiler", "-fPIC", "-shared",
             "--threads", "0", "-I", INCLUDE, "-I", CSRC, "-o", out] + list(extra) + sources())


def _torch():
    """(version, CUDA version or None, directory) of the installed torch, not imported; None without one."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.origin:
        return None
    root = os.path.dirname(spec.origin)
    v = runpy.run_path(os.path.join(root, "version.py"))
    return v["__version__"], v.get("cuda"), root


def _cuda_include():
    """The CUDA toolkit's headers, of nvcc's toolkit or one at a usual place; None without one."""
    nvcc = shutil.which("nvcc")
    roots = [os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))] if nvcc else []
    for root in roots + [r for r in CUDA_ROOTS if r]:
        if os.path.exists(os.path.join(root, "include", "cuda_runtime_api.h")):
            return os.path.join(root, "include")
    return None


def build_binding(force: bool = False) -> str | None:
    """The operators' torch binding; None where there is no torch with CUDA, or no CUDA
    toolkit to build it with (the library and the layer do without it)."""
    torch = _torch()
    if torch is None or torch[1] is None:
        return None
    src = os.path.join(CSRC, "ops_binding.cpp")
    deps = [src] + glob.glob(os.path.join(INCLUDE, "*.h"))
    key = f"{torch[0]} {sysconfig.get_config_var('SOABI')}\n"
    stamp = os.path.splitext(SO_BINDING)[0] + ".stamp"     # the torch and the Python that the file is for
    if not force and os.path.exists(SO_BINDING) and os.path.exists(stamp):
        with open(stamp) as f:
            if f.read() == key and all(os.path.getmtime(d) <= os.path.getmtime(SO_BINDING) for d in deps):
                return SO_BINDING
    cuda = _cuda_include()
    if cuda is None:
        warnings.warn("the operators' torch binding is not built: no CUDA toolkit found (nvcc on the path, CUDA_HOME)")
        return None
    version, _, root = torch
    tmp = SO_BINDING + f".tmp{os.getpid()}"
    subprocess.run(["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f'-DMOE_TORCH_VERSION="{version}"',
                    "-I", INCLUDE, "-I", os.path.join(root, "include"), "-I", cuda,
                    "-I", sysconfig.get_paths()["include"], src, "-o", tmp, "-L", os.path.join(root, "lib"),
                    "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"], check=True)
    if os.path.exists(stamp):
        os.remove(stamp)
    os.replace(tmp, SO_BINDING)
    with open(stamp, "w") as f:
        f.write(key)
    return SO_BINDING


def build(force: bool = False, verbose: bool = False, checked: bool = False) -> str:
    so = SO_CHECKED if checked else SO
    if force or not up_to_date(so):
        tmp = so + f".tmp{os.getpid()}"
        extra = (["-Xptxas", "-v"] if verbose else []) + (["-DMOE_DEBUG_CHECKS"] if checked else [])
        subprocess.run(nvcc_cmd(tmp, extra), check=True)
        os.replace(tmp, so)
    build_binding(force)
    return so


if __name__ == "__main__":
    print(build(force=True, verbose="-v" in sys.argv, checked="--checked" in sys.argv))
