"""Build libtsa.so in-tree with nvcc for sm_103a (no torch extension, no cmake), and tsa_calls.so, the
module that marshals some of its calls, with g++.

    python -m topology_scheduled_gb300.build

Each translation unit compiles in parallel; the library is re-linked only when a source,
header or flag changed (a content hash names the output directory's stamp).
"""
from __future__ import annotations

import hashlib
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libtsa.so")
CALLS = os.path.join(BUILD, "tsa_calls.so")

SOURCES = ["api.cu", "schedule.cu", "segment.cu", "attention.cu", "attention_biased.cu",
           "attention_differential.cu", "terms_api.cu", "backward.cu", "backward_biased.cu", "backward_differential.cu",
           "decode.cu", "rotary.cu", "paged_decode.cu", "cache_api.cu", "noalloc.cu"]
HEADERS = [os.path.join(CSRC, h) for h in ("attention_kernel.cuh", "backward_kernels.cuh", "score_terms.cuh", "tsa_device.cuh",
                                           "tsa_internal.h")] + [os.path.join(INCLUDE, h) for h in ("tsa.h", "tsa_terms.h", "tsa_cache.h")]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
# the CUDA runtime is the one PyTorch has loaded: a second, static one beside it costs 2 us per call
LINK = ARCH + ["-cudart", "shared", "-shared"]
FLAGS = ARCH + ["-lineinfo", "-O3", "-std=c++17", "-Xcompiler", "-fPIC"]
CALLS_FLAGS = ["-O2", "-std=c++17", "-fPIC"]
CALLS_LINK = ["-shared", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-l:libtsa.so", "-Wl,-rpath,$ORIGIN"]


def _calls_flags() -> tuple[list[str], list[str]]:
    """Compiler and linker flags of tsa_calls.so: Python's, PyTorch's and the CUDA runtime's headers."""
    import torch
    home = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    include = [os.path.join(home, "include"), os.path.join(home, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(cuda, "include"), INCLUDE]
    return (CALLS_FLAGS + [f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}"] +
            [x for d in include for x in ("-I", d)],
            ["-L", os.path.join(home, "lib"), "-L", BUILD] + CALLS_LINK)


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libtsa")


def _digest(sources=SOURCES, headers=None, flags=FLAGS + LINK) -> str:
    """Of sources, headers (None: all) and flags, and of no folder: a built tree may be moved, and used where there is no
    compiler."""
    h = hashlib.sha1()
    for p in [os.path.join(CSRC, s) for s in sources] + (HEADERS if headers is None else headers):
        with open(p, "rb") as f:
            h.update(f.read())
    h.update(" ".join(flags).encode())
    return h.hexdigest()[:16]


def _stamped(path: str, stamp: str, digest: str) -> bool:
    """Whether `path` was built from what has this digest."""
    if not os.path.exists(path) or not os.path.exists(stamp):
        return False
    with open(stamp) as f:
        return f.read().strip() == digest


def _linked(cmd: list[str], path: str, stamp: str, digest: str) -> None:
    tmp = f"{path}.{os.getpid()}.tmp"
    r = subprocess.run(cmd + ["-o", tmp], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, path)
    with open(stamp, "w") as f:
        f.write(digest)


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Compile and link libtsa.so, which takes nvcc and its host compiler alone; returns its path."""
    os.makedirs(BUILD, exist_ok=True)
    stamp = os.path.join(BUILD, "stamp")
    digest = _digest()
    if not force and _stamped(LIB, stamp, digest):
        return LIB
    nvcc = _nvcc()

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [nvcc] + FLAGS + ["-I", INCLUDE, "-I", CSRC, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose:
            sys.stderr.write(r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    _linked([nvcc] + LINK + objs, LIB, stamp, digest)
    return LIB


def build_calls(force: bool = False, library=build_library) -> str:
    """Compile tsa_calls.so and link it with libtsa.so (`library` builds that meanwhile); returns its path.  It takes the
    headers of Python, PyTorch and the CUDA runtime, and is for this Python and this PyTorch."""
    import torch
    os.makedirs(BUILD, exist_ok=True)
    stamp, obj = os.path.join(BUILD, "calls.stamp"), os.path.join(BUILD, "calls.o")
    digest = _digest(["calls.cpp"], [os.path.join(INCLUDE, h) for h in ("tsa.h", "tsa_cache.h")],
                     CALLS_FLAGS + CALLS_LINK + [torch.__version__, sys.version])
    if not force and _stamped(CALLS, stamp, digest):
        library()
        return CALLS

    def compile_calls() -> list[str]:
        flags, link = _calls_flags()
        r = subprocess.run(["g++"] + flags + ["-c", os.path.join(CSRC, "calls.cpp"), "-o", obj], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed on calls.cpp:\n{r.stdout}\n{r.stderr}")
        return link

    with ThreadPoolExecutor(max_workers=1) as ex:
        compiled = ex.submit(compile_calls)
        library()
        link = compiled.result()
    _linked(["g++", obj] + link, CALLS, stamp, digest)
    return CALLS


def build(force: bool = False, verbose: bool = False) -> str:
    """Build libtsa.so and tsa_calls.so; returns libtsa.so's path."""
    build_calls(force, lambda: build_library(force, verbose))
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
