"""Build libssm.so (the CUDA library behind include/ssm.h) in-tree with nvcc,
and the Python binding's _marshal module with the C++ compiler.

Every .cu file under csrc/ is compiled for sm_100a and linked into
hybrid_mamba_ssm_b200/libssm.so; csrc/marshal.cpp becomes
hybrid_mamba_ssm_b200/_marshal.so, linked against it and torch.  Run ``python -m hybrid_mamba_ssm_b200.build``
or call ``build()``.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libssm.so")
MARSHAL = os.path.join(HERE, "_marshal.so")
BUILD_DIR = os.path.join(ROOT, "_build")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
              "-Xcompiler", "-fPIC,-fvisibility=hidden", "-I" + os.path.join(ROOT, "include")]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale(target, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile csrc/*.cu into libssm.so (object files go to _build/)."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    nvcc = _nvcc()
    headers = glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) \
        + glob.glob(os.path.join(ROOT, "include", "*.h"))
    objs, cmds = [], []
    for src in sources():
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + headers):
            cmds.append([nvcc, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj])
            if verbose:
                print(" ".join(cmds[-1]), flush=True)
    # one compiler per file at a time, as many as there are cores
    with ThreadPoolExecutor(max_workers=os.cpu_count() or 1) as pool:
        list(pool.map(subprocess.check_call, cmds))
    if force or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.check_call(cmd)
        os.replace(tmp, LIB)
    try:
        build_marshal(force, verbose)
    except (ImportError, OSError, subprocess.CalledProcessError) as e:
        # ssm.py does without it; one of an earlier build may not fit this library
        if os.path.exists(MARSHAL):
            os.remove(MARSHAL)
        warnings.warn(f"_marshal.so could not be built ({e}): calls take more host time", RuntimeWarning, stacklevel=2)
    return LIB


def build_marshal(force: bool = False, verbose: bool = False) -> str:
    """Compile csrc/marshal.cpp into _marshal.so (host code only, for this torch)."""
    import torch
    src = os.path.join(CSRC, "marshal.cpp")
    stamp = os.path.join(BUILD_DIR, "marshal.torch")     # the torch that _marshal.so was built for
    built_for = open(stamp).read() if os.path.exists(stamp) else None
    if not force and built_for == str(torch.__version__) \
            and not _stale(MARSHAL, [src, os.path.join(ROOT, "include", "ssm.h")]):
        return MARSHAL
    os.makedirs(BUILD_DIR, exist_ok=True)
    troot = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    tmp = MARSHAL + f".tmp{os.getpid()}"
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f'-DSSM_TORCH_VERSION="{torch.__version__}"', f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I" + os.path.join(ROOT, "include"), "-isystem", sysconfig.get_paths()["include"],
           "-isystem", os.path.join(troot, "include"),
           "-isystem", os.path.join(troot, "include", "torch", "csrc", "api", "include"), "-isystem", cuda,
           src, "-o", tmp, "-L" + HERE, "-l:libssm.so", "-L" + os.path.join(troot, "lib"), "-ltorch_python",
           "-ltorch_cpu", "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    os.replace(tmp, MARSHAL)
    with open(stamp, "w") as f:
        f.write(torch.__version__)
    return MARSHAL


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True,
          extra_flags=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else [])
