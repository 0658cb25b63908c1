"""Build the in-tree C-ABI library ``libmoe_gb300.so`` with nvcc for sm_103a.

Each ``csrc/*.cu`` translation unit compiles in parallel to an object under
``_build/``; the objects link into one shared library next to this file.
Rebuilds only what changed (source or header newer than the object).
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build", "moe")
LIB = os.path.join(PKG, "libmoe_gb300.so")
# Phase-trace variant of the library (decode kernel with global-timer stamps,
# see trace_phases.py); never loaded by the package unless asked for.
TRACE_BUILD = os.path.join(ROOT, "_build", "moe_trace")
TRACE_LIB = os.path.join(PKG, "libmoe_gb300_trace.so")
# Argument checks of the layer operators in compiled code (see fast_call.cpp); the name
# tells the interpreter, the key what it was compiled for.
FAST_CALL = os.path.join(PKG, "_fast_call" + sysconfig.get_config_var("EXT_SUFFIX"))
FAST_CALL_KEY = os.path.join(ROOT, "_build", "fast_call.key")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    return cand


def _cuda_lib_dir() -> str:
    nvcc = os.path.realpath(_nvcc())
    return os.path.join(os.path.dirname(os.path.dirname(nvcc)), "lib64")


def _newest_dep() -> float:
    deps = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h")) + [__file__]
    return max(os.path.getmtime(d) for d in deps)


def _compile(src: str, extra: list[str], build_dir: str = BUILD) -> str:
    obj = os.path.join(build_dir, os.path.basename(src)[:-3] + ".o")
    if os.path.exists(obj) and os.path.getmtime(obj) >= max(os.path.getmtime(src), _newest_dep()):
        return obj
    cmd = [_nvcc(), *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj + ".tmp"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    os.replace(obj + ".tmp", obj)
    return obj


def build_fast_call() -> str | None:
    """Compile ``csrc/fast_call.cpp`` (host code over PyTorch's headers) into the
    extension module ``_fast_call``, anew where it was compiled for another PyTorch
    or in another way.  Without it (no headers, another compiler, none) the binding
    checks and packs in Python: slower calls, the same kernels; so a failure is
    reported and not raised, and leaves no older module behind."""
    src = os.path.join(CSRC, "fast_call.cpp")
    import torch
    root = os.path.dirname(torch.__file__)
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(_cuda_lib_dir()), "include")]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DMOE_TORCH_VERSION="{torch.__version__}"', "-I", INCLUDE]
    for d in inc:
        cmd += ["-isystem", d]
    lib = os.path.join(root, "lib")
    cmd += [src, "-L", lib, "-Wl,-rpath," + lib, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    key = "\n".join([sys.version, *cmd])
    if os.path.exists(FAST_CALL) and os.path.getmtime(FAST_CALL) >= max(os.path.getmtime(src), _newest_dep()):
        try:
            with open(FAST_CALL_KEY) as f:
                if f.read() == key:
                    return FAST_CALL
        except OSError:
            pass
    for old in (FAST_CALL, os.path.join(os.path.dirname(FAST_CALL), "_fast_call.so")):  # (the name without a tag: once)
        if os.path.exists(old):
            os.remove(old)
    tmp = FAST_CALL + f".tmp{os.getpid()}"
    try:
        r = subprocess.run([*cmd, "-o", tmp], capture_output=True, text=True)
        failed = r.stderr[-2000:] if r.returncode != 0 else None
    except OSError as e:  # no compiler
        failed = str(e)
    if failed is not None:
        print(f"fast_call.cpp was not built (calls are checked in Python instead):\n{failed}", file=sys.stderr)
        return None
    os.replace(tmp, FAST_CALL)
    os.makedirs(os.path.dirname(FAST_CALL_KEY), exist_ok=True)
    with open(FAST_CALL_KEY, "w") as f:
        f.write(key)
    return FAST_CALL


def build(verbose: bool = False, extra: list[str] | None = None, trace: bool = False) -> str:
    """Compile every CUDA source and link the shared library; returns its path.
    ``trace=True`` builds the phase-trace variant (``-DMOE_PHASE_TRACE``) into
    its own directory and library instead."""
    build_dir, lib = (TRACE_BUILD, TRACE_LIB) if trace else (BUILD, LIB)
    os.makedirs(build_dir, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    extra = list(extra or []) + (["-DMOE_PHASE_TRACE"] if trace else [])
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs)) + 1) as ex:
        fast = None if trace else ex.submit(build_fast_call)
        objs = list(ex.map(lambda s: _compile(s, extra, build_dir), srcs))
        if fast is not None:
            fast.result()
    newest = max(os.path.getmtime(o) for o in objs)
    if not os.path.exists(lib) or os.path.getmtime(lib) < newest:
        tmp = lib + f".tmp{os.getpid()}"
        cmd = [_nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "shared",
               "-Xlinker", "-rpath," + _cuda_lib_dir()]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, lib)
    if verbose:
        print(lib)
    return lib


def ptxas_report() -> str:
    """Registers / spills / shared memory per kernel (``-Xptxas -v``)."""
    out = []
    for src in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        cmd = [_nvcc(), *ARCH, *NVCC_FLAGS, "-Xptxas", "-v", "-c", src, "-o", os.devnull]
        r = subprocess.run(cmd, capture_output=True, text=True)
        out.append(f"== {os.path.basename(src)}\n{r.stderr}")
    return "\n".join(out)


if __name__ == "__main__":
    build(verbose=True)
