"""Build the HIP library ``_kda.so`` (gfx950) and the binding's ``_kda_marshal.so`` in-tree.

Every source under ``csrc/`` is compiled for gfx950 only.  Packed-fp32 instructions are
disabled (``-packed-fp32-ops``).  The library links the HIP runtime by soname, so when
loaded after ``import torch`` it shares torch's runtime (one HIP runtime per process).
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "_kda.so")
MARSHAL = os.path.join(PKG, "_kda_marshal.so")
ARCH = "gfx950"


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found")


def compile_flags() -> list:
    return [
        f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-Wall", "-Wno-unused-function",
        "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
        "-I", INCLUDE, "-I", CSRC,
    ]


def build_library(verbose: bool = False, jobs: int = 8) -> str:
    """Compile csrc/*.hip and csrc/*.cpp to objects (in parallel), link ``_kda.so``."""
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.hip")) + glob.glob(os.path.join(CSRC, "*.cpp")))
    objdir = os.path.join(PKG, "_build")
    os.makedirs(objdir, exist_ok=True)
    procs, objs = [], []
    for s in srcs:
        o = os.path.join(objdir, os.path.basename(s) + ".o")
        objs.append(o)
        cmd = [hipcc()] + compile_flags() + ["-c", s, "-o", o]
        if s.endswith(".cpp"):
            cmd = [hipcc(), "-x", "hip"] + compile_flags() + ["-c", s, "-o", o]
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((s, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
        if len(procs) >= jobs:
            _wait(procs.pop(0))
    for p in procs:
        _wait(p)
    tmp = LIB + ".tmp"
    cmd = [hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp] + objs
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


def build_marshal(verbose: bool = False):
    """Compile binding/kda_marshal.cpp (host code against torch's headers) to ``_kda_marshal.so``.

    Returns its path, or None where there is no g++ or a header is missing: the binding then marshals in
    Python, with the same results."""
    import sysconfig

    import torch

    base = os.path.dirname(torch.__file__)
    python = sysconfig.get_paths()["include"]
    missing = [] if shutil.which("g++") else ["g++"]
    missing += [h for h in (os.path.join(python, "Python.h"),
                            os.path.join(base, "include", "torch", "csrc", "autograd", "python_variable.h"))
                if not os.path.exists(h)]
    if missing:
        if os.path.exists(MARSHAL):  # it may not fit the library that has just been built
            os.remove(MARSHAL)
        print(f"{os.path.basename(MARSHAL)} not built (no {', '.join(missing)}); the calls are marshalled in Python",
              flush=True)
        return None
    tmp = MARSHAL + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", INCLUDE, "-isystem", os.path.join(base, "include"),
           "-isystem", os.path.join(base, "include", "torch", "csrc", "api", "include"),
           f'-DKDA_TORCH_VERSION="{torch.__version__}"',
           "-isystem", python, os.path.join(PKG, "binding", "kda_marshal.cpp"), "-o", tmp,
           "-L", os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, MARSHAL)
    return MARSHAL


def _wait(item):
    src, p = item
    out, _ = p.communicate()
    text = out.decode(errors="replace")
    if p.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{text}")
    lines = [ln for ln in text.splitlines() if "packed-fp32-ops" not in ln]
    if any(lines):
        print("\n".join(lines), flush=True)


if __name__ == "__main__":
    print(build_library(verbose=True))
    print(build_marshal(verbose=True))
