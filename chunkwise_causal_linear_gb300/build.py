"""Builds liblachunked.so (the CUDA kernels and the C ABI) in-tree for sm_103a, and _layer.so (the
torch-tensor binding of the operators around the attention).

    python -m chunkwise_causal_linear_gb300.build [--force] [--verbose]

Each .cu file is compiled on its own (in parallel) with nvcc for sm_103a only, then
linked into chunkwise_causal_linear_gb300/liblachunked.so.  binding.cpp is compiled with g++
against the installed torch (one with CUDA) and linked with that library into _layer.so; another torch
or Python builds it again.
"""
from __future__ import annotations

import importlib.util
import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "liblachunked.so")
LAYER = os.path.join(HERE, "_layer.so")
STAMP = os.path.join(BUILD, "binding.stamp")  # what _layer.so was built against


def cuda_torch(path):
    """The torch to bind to: None without one that has CUDA, and then the C ABI alone is built."""
    return path if path and os.path.exists(os.path.join(path, "lib", "libc10_cuda.so")) else None


_spec = importlib.util.find_spec("torch")
TORCH = cuda_torch(os.path.dirname(_spec.origin) if _spec else None)
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
SOURCES = ["api.cu", "simt.cu", "tc.cu", "tc_favor.cu", "tc_loglinear.cu", "tc_wide.cu", "decode.cu", "noncausal.cu", "noalloc.cu", "bwd.cu", "bwd_ll.cu",
           "recurrence.cu", "rotary.cu", "group_norm.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE]


def _deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "la_chunked.h"))
    files.append(os.path.abspath(__file__))
    return files


def binding_stamp() -> str:
    """The torch (place and version) and the Python that a binding built now is for."""
    with open(os.path.join(TORCH, "version.py")) as f:
        version = f.read()
    return f"{TORCH}\n{sysconfig.get_config_var('SOABI')}\n{version}"


def _read(path):
    try:
        with open(path) as f:
            return f.read()
    except OSError:
        return None


def up_to_date() -> bool:
    libs = [LIB, LAYER] if TORCH else [LIB]
    if not all(os.path.exists(f) for f in libs):
        return False
    if TORCH and _read(STAMP) != binding_stamp():
        return False
    t = min(os.path.getmtime(f) for f in libs)
    return all(os.path.getmtime(f) <= t for f in _deps())


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [NVCC, *ARCH, *FLAGS, *extra_flags, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, flush=True)
        return obj

    def run(cmd, what):
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")

    def compile_binding():
        obj = os.path.join(BUILD, "binding.o")
        dirs = [INCLUDE, sysconfig.get_paths()["include"], os.path.join(TORCH, "include"),
                os.path.join(TORCH, "include", "torch", "csrc", "api", "include"),
                os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include")]
        run(["g++", "-O2", "-std=c++17", "-fPIC", *(f"-I{d}" for d in dirs), "-c",
             os.path.join(CSRC, "binding.cpp"), "-o", obj], "g++ on binding.cpp")
        return obj

    with ThreadPoolExecutor(len(SOURCES) + 1) as ex:
        binding = ex.submit(compile_binding) if TORCH else None
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + f".{os.getpid()}.tmp"
    cmd = [NVCC, *ARCH, "-shared", "-o", tmp, *objs, "-L/usr/local/cuda/lib64/stubs", "-lcuda"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if binding is None:
        return LIB
    # the library and torch's are found beside _layer.so and where torch is installed
    tmp, torch_lib = LAYER + f".{os.getpid()}.tmp", os.path.join(TORCH, "lib")
    run(["g++", "-shared", "-o", tmp, binding.result(), f"-L{HERE}", "-l:" + os.path.basename(LIB),
         "-Wl,-rpath,$ORIGIN", f"-L{torch_lib}", f"-Wl,-rpath,{torch_lib}", "-ltorch", "-ltorch_cpu",
         "-ltorch_python", "-lc10", "-lc10_cuda"], "link of _layer.so")
    os.replace(tmp, LAYER)
    with open(STAMP, "w") as f:
        f.write(binding_stamp())
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="--verbose" in sys.argv)
    print(LIB)
