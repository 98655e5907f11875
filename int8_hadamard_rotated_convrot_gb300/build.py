"""Builds libconvrot.so in-tree with nvcc for sm_103a.

Each .cu file under csrc/ and csrc16/ compiles to an object in parallel, then nvcc links
them into ``_build/libconvrot.so`` next to this file, and the CPython module of
csrc/block_py.cpp (g++, the installed torch's headers) is linked to it. Rebuilds only when a
source or header is newer than the library.
"""

from __future__ import annotations

import concurrent.futures
import glob
import os
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
CSRC16 = os.path.join(HERE, "csrc16")  # attention and the gated linear, on 16-bit tensors
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libconvrot.so")
# the CPython module that marshals block.py's tensors (csrc/block_py.cpp), linked to LIB
BLOCK_SOURCE = os.path.join(CSRC, "block_py.cpp")
BLOCK_MODULE = os.path.join(BUILD, "_block" + sysconfig.get_config_var("EXT_SUFFIX"))

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE,
         "--expt-relaxed-constexpr"]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found")
    return path


def _sources():
    return sorted(p for d in (CSRC, CSRC16) for p in glob.glob(os.path.join(d, "*.cu")))


def _deps():
    return (_sources() + [p for d in (CSRC, CSRC16) for e in ("*.h", "*.cuh") for p in glob.glob(os.path.join(d, e))]
            + glob.glob(os.path.join(INCLUDE, "*.h")) + [BLOCK_SOURCE, os.path.abspath(__file__)])


def up_to_date() -> bool:
    if not (os.path.exists(LIB) and os.path.exists(BLOCK_MODULE)):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(BLOCK_MODULE))
    return all(os.path.getmtime(p) <= t for p in _deps())


def _compile_block_object() -> str:
    """csrc/block_py.cpp against the headers of the installed torch, with the host compiler."""
    import torch

    base = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    obj = os.path.join(BUILD, "block_py.o")
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-w", "-I", sysconfig.get_paths()["include"],
           "-I", os.path.join(base, "include"), "-I", os.path.join(base, "include", "torch", "csrc", "api", "include"),
           "-I", cuda, f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-c", BLOCK_SOURCE, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {BLOCK_SOURCE}:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_block_module(obj: str) -> None:
    import torch

    # libconvrot.so is found next to the module, torch's libraries where torch loads them from
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BLOCK_MODULE + f".tmp{os.getpid()}"
    cmd = [shutil.which("g++") or "g++", "-shared", "-o", tmp, obj, "-L", BUILD, "-lconvrot", "-L", libs, "-ltorch_python",
           "-ltorch_cpu", "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + libs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of the block module failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BLOCK_MODULE)


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    extra = list(extra or [])

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [cc, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    with concurrent.futures.ThreadPoolExecutor(max_workers=12) as ex:
        block_obj = ex.submit(_compile_block_object)
        objs = list(ex.map(compile_one, _sources()))
        block_obj = block_obj.result()
    tmp = LIB + f".tmp{os.getpid()}"
    r = subprocess.run([cc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    _link_block_module(block_obj)
    return LIB


if __name__ == "__main__":
    import sys

    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                extra=["-Xptxas", "-v"] if "--ptxas" in sys.argv else None))
