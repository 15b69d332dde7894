"""Build the CUDA library libmoe_b200.so in-tree with nvcc for sm_100a, and the
Python extension _binding.so (csrc/binding.cpp) against it.

    python -m bit_quantized_mixture_b200.build [--force] [--verbose] [--library-only]

Objects go to bit_quantized_mixture_b200/_build/; the shared library is
written next to this file so that it travels with the source tree.
"""
from __future__ import annotations

import argparse
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmoe_b200.so")
INCLUDE = os.path.join(ROOT, "include")
BINDING = os.path.join(PKG, "_binding.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
STAMP = os.path.join(BUILD, "binding.stamp")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC",
         "-Xcompiler", "-Wall", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hs += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    return hs


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def binding_command(target):
    """g++ command of the Python extension (host code; tensors through torch's C++ headers)."""
    import torch
    troot = os.path.dirname(torch.__file__)
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    cmd += ["-I" + INCLUDE, "-isystem", os.path.join(troot, "include"), "-isystem", os.path.join(troot, "include", "torch", "csrc", "api", "include")]
    cmd += ["-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
    cmd += [BINDING_SRC, "-o", target, "-L" + PKG, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN"]
    cmd += ["-L" + os.path.join(troot, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    return cmd


def binding_missing():
    """What the extension cannot be compiled without and is not here, or None."""
    if not shutil.which("g++"):
        return "g++ was not found"
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "Python's headers were not found"
    try:
        import torch
    except ImportError:
        return "torch cannot be imported"
    if not os.path.exists(os.path.join(os.path.dirname(torch.__file__), "include", "torch", "csrc", "autograd", "python_variable.h")):
        return "torch's C++ headers were not found"
    return None


def binding_stamp() -> str:
    """What the extension is compiled against: it fits this Python and this torch only."""
    import torch
    return "\n".join([sys.version, torch.__version__] + binding_command(BINDING)) + "\n"


def build(force: bool = False, verbose: bool = False, extra=None, binding: bool = True) -> str:
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    hdrs = headers()
    objs, jobs = [], []
    for src in sources():
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + hdrs + [__file__]):
            cmd = [cc] + ARCH + FLAGS + (extra or []) + ["-c", src, "-o", obj]
            jobs.append(cmd)

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{os.path.basename(cmd[0])} failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, flush=True)

    with ThreadPoolExecutor(max(1, min(len(jobs), os.cpu_count() or 4))) as ex:
        list(ex.map(run, jobs))
    if force or jobs or _stale(LIB, objs):
        cmd = [cc] + ARCH + ["-shared", "-o", LIB + ".tmp"] + objs + ["-lcudart"]
        run(cmd)
        os.replace(LIB + ".tmp", LIB)
    if not binding:
        return LIB
    # the library is complete by itself: its C callers need nothing of what the
    # extension is compiled with
    missing = binding_missing()
    if missing:
        print(f"_binding.so is not built: {missing}; the library's C interface does not need it, the Python calls around the experts do",
              file=sys.stderr, flush=True)
        return LIB
    stamp, made = binding_stamp(), None
    if os.path.exists(STAMP):
        with open(STAMP) as f:
            made = f.read()
    # the entry points' declarations and the extension's own source (the library
    # is found by name when it is loaded)
    if force or made != stamp or _stale(BINDING, [BINDING_SRC, os.path.join(INCLUDE, "moe_b200.h"), __file__]):
        run(binding_command(BINDING + ".tmp"))
        os.replace(BINDING + ".tmp", BINDING)
        with open(STAMP, "w") as f:
            f.write(stamp)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--library-only", action="store_true", help="the C library without the Python extension")
    ap.add_argument("--ptxas-info", action="store_true", help="print register/smem usage per kernel")
    a = ap.parse_args()
    extra = ["-Xptxas", "-v"] if a.ptxas_info else None
    print(build(force=a.force or a.ptxas_info, verbose=a.verbose or a.ptxas_info, extra=extra, binding=not a.library_only))
    sys.exit(0)
