"""Build libshampoo4.so in-tree with nvcc for sm_100a:

    python -m bit_quantized_shampoo_b200.build [--force] [-v]

and beside it _act8.so, the Python binding of the 8-bit activation calls
(g++, against this interpreter and its torch; where their headers are missing
the library is built alone, and the act8 calls say so).
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libshampoo4.so")

SOURCES = ["quant4.cu", "gemm_simt.cu", "gemm_tc.cu", "kernels_misc.cu", "graft.cu", "shampoo4.cu", "noalloc.cu",
           "act8.cu", "act8_grad.cu", "act8_gemm.cu"]
BINDING = os.path.join(PKG, "_act8.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
         "-Xcompiler", "-fPIC", "-I" + INCLUDE, "-I" + CSRC]


def _headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hs.append(os.path.join(INCLUDE, "shampoo4.h"))
    return hs


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    headers = _headers()
    objs, jobs = [], []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s] + headers):
            jobs.append([NVCC, *FLAGS, "-c", s, "-o", o])

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{os.path.basename(cmd[0])} failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        return r

    with concurrent.futures.ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        list(ex.map(run, jobs))
    if force or jobs or _stale(LIB, objs):
        run([NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-o", LIB, *objs,
             "-lcudart_static", "-lrt", "-ldl", "-lpthread"])
    _build_binding(run, force)
    return LIB


def _build_binding(run, force):
    """The binding, rebuilt when its sources change or its command does (which
    names the interpreter and the torch that it is for)."""
    missing = _binding_missing()
    if missing:
        if os.path.exists(BINDING):
            os.remove(BINDING)                    # made for another interpreter or torch
        print(f"_act8.so is not built: {missing}; the act8 calls of api.py will not work", file=sys.stderr)
        return
    src = os.path.join(CSRC, "act8_binding.cpp")
    cmd = _binding_command(src)
    stamp = os.path.join(BUILD, "act8_binding.command")
    text = "\n".join(cmd)
    same = os.path.exists(stamp) and open(stamp).read() == text
    if force or not same or _stale(BINDING, [src, os.path.join(INCLUDE, "shampoo4.h")]):
        run(cmd)
        with open(stamp, "w") as f:
            f.write(text)


def _binding_missing():
    """What the binding needs and this machine does not have, or None."""
    import importlib.util
    import sysconfig
    cxx = os.environ.get("CXX", "g++")
    if not shutil.which(cxx.split()[0]):
        return f"no compiler {cxx}"
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "no Python.h"
    spec = importlib.util.find_spec("torch")
    if spec is None or not os.path.isdir(os.path.join(os.path.dirname(spec.origin), "include", "ATen")):
        return "no torch headers"
    return None


def _binding_command(src):
    """The g++ command of the binding.  Its C entry points come from
    libshampoo4.so beside it, the rest from the torch that loads it."""
    import sysconfig
    import torch
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(NVCC))
    flags = ["-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
             f'-DACT8_BUILT_FOR="{torch.__version__}"']
    inc = [INCLUDE, sysconfig.get_paths()["include"], os.path.join(base, "include"),
           os.path.join(base, "include", "torch", "csrc", "api", "include"), os.path.join(cuda, "include")]
    return [*os.environ.get("CXX", "g++").split(), *flags, *[f"-I{i}" for i in inc], src, "-o", BINDING,
            f"-L{PKG}", "-l:libshampoo4.so", "-Wl,-rpath,$ORIGIN", f"-L{os.path.join(base, 'lib')}",
            "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
