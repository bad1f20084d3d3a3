"""Builds libdflash_gb300.so in-tree with nvcc for sm_103a (GB300) only.

Translation units are compiled in parallel, then linked with nvcc -shared. The output
lands in speculative_decoding_draft_rmsnorm_gb300/_lib/; objects go to _build/.

A second library, libdflash_gb300_waittest.so, is built from the same sources with
DFLASH_WAIT_TEST defined: device waits give up after 5 ms instead of 2 s, and hooks can
withhold one copy of a kernel, so that a test can watch a bounded wait run out and the
kernel unwind. Only the tests load it; the package loads the product library.

The marshalling module of decode.py (csrc/bind.cpp, host C++ against torch and the product
library) is built last, and only decode.py's calls need it: the libraries build and load
without torch.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJ_DIR = os.path.join(PKG, "_build")
LIB_DIR = os.path.join(PKG, "_lib")
LIB_NAME = "libdflash_gb300.so"
LIB_PATH = os.path.join(LIB_DIR, LIB_NAME)
SOURCES = ["api.cu", "attention.cu", "norm_rope.cu", "noalloc.cu", "draft_step.cu", "rotary.cu",
           "decode_attention.cu", "beam.cu", "pages.cu", "rms_norm.cu", "shared_prefixes.cu",
           "shared_attention.cu"]
HEADERS = ["ptx.cuh", "internal.h", "norm_rope.cuh", "decode_host.h", "attention_parts.cuh"]
# The marshalling module of decode.py: host C++ against torch and the product library.
BIND_SOURCE = os.path.join(CSRC, "bind.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "-DDFLASH_BUILD"]


def nvcc() -> str:
    p = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(p):
        raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build the library")
    return p


def bind_path() -> str:
    """The marshalling module. It uses parts of torch that change between versions: the file is named after the
    interpreter, the torch and the C++ ABI that it was built for."""
    import sysconfig

    import torch
    return os.path.join(LIB_DIR, f"_decode_bind.{sysconfig.get_config_var('SOABI')}-torch{torch.__version__}"
                                 f"-abi{int(torch._C._GLIBCXX_USE_CXX11_ABI)}.so")


WAIT_TEST_LIB_PATH = os.path.join(LIB_DIR, "libdflash_gb300_waittest.so")
# (library, extra nvcc flags, object folder)
TARGETS = [(LIB_PATH, [], OBJ_DIR),
           (WAIT_TEST_LIB_PATH, ["-DDFLASH_WAIT_TEST"], os.path.join(OBJ_DIR, "waittest"))]


def _inputs() -> list[str]:
    files = [os.path.join(CSRC, s) for s in SOURCES + HEADERS]
    files.append(os.path.join(ROOT, "include", "dflash.h"))
    return files


def up_to_date(path: str = LIB_PATH) -> bool:
    """Whether a library (or the marshalling module) is there and newer than its sources."""
    if not os.path.exists(path):
        return False
    t = os.path.getmtime(path)
    bind = os.path.basename(path).startswith("_decode_bind.")
    files = [BIND_SOURCE, os.path.join(ROOT, "include", "dflash.h")] if bind else _inputs()
    return all(os.path.getmtime(f) <= t for f in files)


def _compile_bind() -> str:
    """bind.cpp to an object (the library it links to is not needed yet)."""
    import sysconfig

    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    obj = os.path.join(OBJ_DIR, "bind.o")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I" + inc,
           "-I" + os.path.join(inc, "torch", "csrc", "api", "include"), "-I" + sysconfig.get_paths()["include"], "-I" + cuda,
           "-c", BIND_SOURCE, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on bind.cpp:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_bind(obj: str) -> None:
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    path = bind_path()
    tmp = path + f".tmp{os.getpid()}"
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L" + lib, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda",
           "-L" + LIB_DIR, "-l:" + LIB_NAME, "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"linking the marshalling module failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, path)


def build(force: bool = False, verbose: bool = False, bind: bool = True) -> str:
    """Builds both libraries (every translation unit of both in one parallel pass) and, unless
    bind is False, the marshalling module; returns the product library's path."""
    todo = [t for t in TARGETS if force or not up_to_date(t[0])]
    bind = bind and (force or not up_to_date(bind_path()))
    if not todo and not bind:
        return LIB_PATH
    os.makedirs(LIB_DIR, exist_ok=True)
    os.makedirs(OBJ_DIR, exist_ok=True)
    cc = nvcc()

    def compile_one(job) -> str:
        src, extra, obj_dir = job
        obj = os.path.join(obj_dir, src.replace(".cu", ".o"))
        cmd = [cc, *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src} {' '.join(extra)}:\n{r.stdout}\n{r.stderr}")
        if verbose:
            print(r.stdout + r.stderr)
        return obj

    jobs = []
    for _, extra, obj_dir in todo:
        os.makedirs(obj_dir, exist_ok=True)
        jobs += [(src, extra, obj_dir) for src in SOURCES]
    workers = max(1, min(len(jobs) + bind, os.cpu_count() or 1))
    with cf.ThreadPoolExecutor(workers) as ex:
        bind_obj = ex.submit(_compile_bind) if bind else None
        objs = list(ex.map(compile_one, jobs))
    for i, (path, _, _) in enumerate(todo):
        tmp = path + f".tmp{os.getpid()}"
        mine = objs[i * len(SOURCES):(i + 1) * len(SOURCES)]
        r = subprocess.run([cc, *ARCH, "-shared", "-o", tmp, *mine, "-lcudart"], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, path)
    if bind:
        _link_bind(bind_obj.result())  # its failure leaves the libraries built
    return LIB_PATH


if __name__ == "__main__":
    print(build(force=True, verbose=True))
