"""Builds libpa.so (the C-ABI CUDA library) in-tree for sm_103a with nvcc, and
the extension module _pa_call.so with g++.

Each translation unit compiles in its own nvcc process (in parallel), then
they link into ``paged_kv_cache_72_gb300/libpa.so`` with the CUDA runtime
linked statically, so the library needs no CUDA driver to be loaded (it finds
the driver at run time).  That takes nvcc alone: ``build_library()``, and this
file run as a script where torch is not installed.  ``_pa_call.so`` (the Python
side of some calls, host code only) is linked against the library and against
the installed torch; the library is in place before that, whatever becomes of it.
"""
import hashlib
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build", "libpa")
LIB = os.path.join(PKG, "libpa.so")
CALL = os.path.join(PKG, "_pa_call.so")

SOURCES = ["pa_api.cu", "pa_append.cu", "pa_cache_ops.cu", "pa_decode_fp4.cu", "pa_decode.cu",
           "pa_decode_d64.cu", "pa_decode_d128.cu", "pa_decode_f8_d64.cu", "pa_decode_f8_d128.cu", "pa_decode_noalloc.cu", "pa_prefill.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I" + INCLUDE]


def _nvcc():
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found")
    return exe


def _torch_dir():
    import torch
    return os.path.dirname(torch.__file__), torch.__version__


CALL_SOURCE = "pa_call.cpp"


def _files(library):
    """Sources of the library, or of the extension module."""
    if not library:
        return [os.path.join(CSRC, CALL_SOURCE), os.path.join(INCLUDE, "pa.h")]
    paths = [os.path.join(d, name) for d in (CSRC, INCLUDE) for name in sorted(os.listdir(d))]
    return [p for p in paths if os.path.isfile(p) and os.path.basename(p) != CALL_SOURCE]


def _digest(library, *more):
    h = hashlib.sha256()
    for p in _files(library):
        h.update(os.path.basename(p).encode())
        with open(p, "rb") as f:
            h.update(f.read())
    h.update(" ".join(more).encode())
    return h.hexdigest()


def _current(product, stamp, digest):
    if not os.path.exists(product) or not os.path.exists(stamp):
        return False
    with open(stamp) as f:
        return f.read().strip() == digest


def _run(cmd, what, verbose=False):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("%s failed:\n%s%s" % (what, r.stdout, r.stderr))
    if verbose:
        sys.stderr.write(r.stderr)


def build_library(force=False, verbose=False):
    """Compile libpa.so (if sources changed) and return its path."""
    os.makedirs(BUILD, exist_ok=True)
    stamp = os.path.join(BUILD, "digest")
    dig = _digest(True, *ARCH, *FLAGS)
    if not force and _current(LIB, stamp, dig):
        return LIB
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [nvcc] + ARCH + FLAGS + ["-c", os.path.join(CSRC, src), "-o", obj]
        _run(cmd + (["-Xptxas=-v"] if verbose else []), "nvcc for " + src, verbose)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + ".tmp%d" % os.getpid()
    _run([nvcc] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs, "linking libpa.so")
    os.replace(tmp, LIB)
    with open(stamp, "w") as f:
        f.write(dig)
    return LIB


def build_call(force=False, library=build_library):
    """Compile _pa_call.so (if its source, torch or Python changed) and return
    its path; `library` is called for libpa.so before the link."""
    os.makedirs(BUILD, exist_ok=True)
    torch_dir, torch_version = _torch_dir()
    stamp = os.path.join(BUILD, "digest_call")
    dig = _digest(False, torch_version, sys.version)
    if not force and _current(CALL, stamp, dig):
        return CALL
    cuda_dir = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    obj = os.path.join(BUILD, "pa_call.o")
    inc = [os.path.join(torch_dir, "include"),
           os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda_dir, "include")]
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-c", os.path.join(CSRC, CALL_SOURCE), "-o", obj]
         + ["-I" + d for d in inc], "g++ for " + CALL_SOURCE)
    library()
    tmp = CALL + ".tmp%d" % os.getpid()
    lib = os.path.join(torch_dir, "lib")
    _run(["g++", "-shared", "-o", tmp, obj, "-L" + PKG, "-lpa", "-L" + lib, "-ltorch_python",
          "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib],
         "linking _pa_call.so")
    os.replace(tmp, CALL)
    with open(stamp, "w") as f:
        f.write(dig)
    return CALL


def build(force=False, verbose=False):
    """Compile both (what changed), and return the path of libpa.so."""
    with ThreadPoolExecutor(max_workers=2) as ex:
        lib = ex.submit(build_library, force, verbose)
        call = ex.submit(build_call, force, lib.result)
        lib.result()
        call.result()
    return LIB


if __name__ == "__main__":
    args = dict(force="--force" in sys.argv, verbose="-v" in sys.argv)
    if importlib.util.find_spec("torch") is None:
        sys.stderr.write("torch is not installed: libpa.so alone\n")
        print(build_library(**args))
    else:
        print(build(**args))
