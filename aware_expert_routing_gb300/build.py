"""Builds libaware_moe.so (the C-ABI library) in-tree with nvcc for sm_103a.

Each .cu file is compiled in parallel, then linked into one shared library
next to this file; binding.cpp becomes the extension module _binding.so,
which links to it.  The library needs nvcc only: without g++ on the path, torch
or Python's headers the module is left out, which callers of the C ABI do
without.  Set MOE_PTXAS_VERBOSE=1 to print register and shared memory usage per
kernel.
"""
from __future__ import annotations

import concurrent.futures
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libaware_moe.so")
BINDING = os.path.join(HERE, "_binding.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
SOURCES = ["api.cu", "router.cu", "route.cu", "ffn_tc.cu", "ffn_f32.cu", "synth.cu", "pack.cu", "residency.cu",
           "static_scratch.cu", "rope.cu", "attention.cu",
           "attention_tc.cu"]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found")
    return path


def binding_lacks() -> str:
    """What building the extension module wants and this machine has not."""
    if not shutil.which("g++"):
        return "g++"
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "Python.h"
    return "" if importlib.util.find_spec("torch") else "torch"


def compile_binding(obj: str):
    """binding.cpp with the host compiler, against Python's, torch's and
    CUDA's headers.  Returns the folder of torch's libraries; raises if the
    code does not compile."""
    torch_dir = os.path.dirname(importlib.util.find_spec("torch").origin)
    inc = [sysconfig.get_paths()["include"], os.path.join(torch_dir, "include"),
           os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
           os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include"), os.path.join(HERE, "..", "include")]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-w", "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj]
    r = subprocess.run(cmd + [x for i in inc for x in ("-isystem", i)], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on binding.cpp:\n{r.stdout}\n{r.stderr}")
    return os.path.join(torch_dir, "lib")


def _deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(HERE, "..", "include", "moe.h"))
    return files


def up_to_date() -> bool:
    made = [LIB] if binding_lacks() else [LIB, BINDING]
    if not all(os.path.exists(f) for f in made):
        return False
    t = min(os.path.getmtime(f) for f in made)
    return all(os.path.getmtime(f) <= t for f in _deps() + [__file__])


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
                    "-I" + os.path.join(HERE, "..", "include")]
    if verbose or os.environ.get("MOE_PTXAS_VERBOSE"):
        flags += ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [nvcc()] + flags + ["-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if r.stderr.strip() and (verbose or os.environ.get("MOE_PTXAS_VERBOSE")):
            sys.stderr.write(r.stderr)
        return obj

    bind = os.path.join(BUILD, "binding.o")
    lacks = binding_lacks()
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = None if lacks else ex.submit(compile_binding, bind)
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc()] + ARCH + ["-shared", "-Xlinker", "-soname," + os.path.basename(LIB), "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    # the library stands, whatever becomes of the module
    if lacks:
        sys.stderr.write(f"{os.path.basename(BINDING)} left out (the per-token Python calls need it): no {lacks}\n")
        return LIB
    torch_lib = binding.result()
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = ["g++", "-shared", "-o", tmp, bind, "-L" + HERE, "-l:" + os.path.basename(LIB), "-L" + torch_lib,
           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN",
           "-Wl,-rpath," + torch_lib]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
