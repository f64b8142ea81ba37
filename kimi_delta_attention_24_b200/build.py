"""Builds libkda_b200.so (the C-ABI library) in-tree with nvcc for sm_100a, and attn_binding.*.so, the
Python binding of its softmax-attention operators, with g++ against torch's headers.  The binding is
linked against torch's C++ libraries, so the versions of torch and Python are part of its file name: a
binding built for others is never loaded.  The C library needs neither.

    python -m kimi_delta_attention_24_b200.build [--force]
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_DIR = os.path.join(PKG, "lib")
LIB_PATH = os.path.join(LIB_DIR, "libkda_b200.so")

SOURCES = ["kda_api.cu", "kda_recurrent.cu", "kda_chunked.cu", "kda_split.cu", "kda_fwd_static.cu",
           "kda_selftest.cu", "kda_decode.cu", "kda_kcp.cu", "kda_bwd.cu", "kda_pad.cu",
           "attn_api.cu", "attn_cache.cu", "attn_decode.cu"]
BINDING_SRC = os.path.join(CSRC, "attn_binding.cpp")
ARCH_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ARCH_FLAGS + ["-lineinfo", "-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
                           f"-I{INCLUDE}", f"-I{CSRC}"]


def _nvcc() -> str:
    cuda_home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    cand = os.path.join(cuda_home, "bin", "nvcc")
    return cand if os.path.exists(cand) else (shutil.which("nvcc") or "nvcc")


def _deps() -> list:
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    return headers + [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]


def _stale(target: str, inputs) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(i) > t for i in inputs)


def _torch() -> tuple:
    """The folder and the version of the installed torch, found without importing it."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.origin:
        raise RuntimeError("attn_binding is built against torch, which is not installed")
    folder = os.path.dirname(spec.origin)
    with open(os.path.join(folder, "version.py")) as f:
        return folder, re.search(r"^__version__ = ['\"](.+)['\"]", f.read(), re.M).group(1)


def binding_path() -> str:
    """Where the binding for this torch and this Python is."""
    return os.path.join(LIB_DIR, f"attn_binding.torch-{_torch()[1]}{sysconfig.get_config_var('EXT_SUFFIX')}")


def _binding_command(out: str) -> list:
    """g++ for the binding: torch's headers and libraries."""
    torch_dir = _torch()[0]
    cuda_home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    inc = [os.path.join(torch_dir, "include"), os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda_home, "include"), sysconfig.get_paths()["include"]]
    lib = os.path.join(torch_dir, "lib")
    return (["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", f"-I{INCLUDE}"] + [x for p in inc for x in ("-isystem", p)]
            + [BINDING_SRC, "-o", out, f"-L{lib}", f"-Wl,-rpath,{lib}", "-lc10", "-lc10_cuda", "-ltorch", "-ltorch_cpu",
               "-ltorch_cuda", "-ltorch_python"])


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    os.makedirs(LIB_DIR, exist_ok=True)
    nvcc = _nvcc()
    deps = _deps()
    objs = []
    jobs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s] + deps + [__file__]):
            jobs.append([nvcc] + NVCC_FLAGS + ["-c", s, "-o", o])

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"the compiler failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)

    def bind():
        path = binding_path()
        if force or _stale(path, [BINDING_SRC, __file__, os.path.join(INCLUDE, "kda.h")]):
            tmp = path + f".tmp{os.getpid()}"
            run(_binding_command(tmp))
            os.replace(tmp, path)

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(bind)
        list(ex.map(run, jobs))
    if force or jobs or _stale(LIB_PATH, objs):
        tmp = LIB_PATH + f".tmp{os.getpid()}"
        run([nvcc] + ARCH_FLAGS + ["-shared", "-o", tmp] + objs)
        os.replace(tmp, LIB_PATH)
    binding.result()  # (its failure is raised when the C library, which does not need it, is in its place)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
