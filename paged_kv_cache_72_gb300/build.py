"""Builds libpa.so (the C-ABI CUDA library) in-tree for sm_103a with nvcc, and
the extension module _pa_call.so with g++.

Each translation unit compiles in its own nvcc process (in parallel), then
they link into ``paged_kv_cache_72_gb300/libpa.so`` with the CUDA runtime
linked statically, so the library needs no CUDA driver to be loaded (it finds
the driver at run time).  ``_pa_call.so`` (the Python side of some calls, host
code only) is linked against it and against the installed torch.
"""
import hashlib
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


def _digest():
    h = hashlib.sha256()
    h.update((_torch_dir()[1] + sys.version).encode())
    for d in (CSRC, INCLUDE):
        for name in sorted(os.listdir(d)):
            p = os.path.join(d, name)
            if os.path.isfile(p):
                h.update(name.encode())
                with open(p, "rb") as f:
                    h.update(f.read())
    h.update(" ".join(ARCH + FLAGS).encode())
    return h.hexdigest()


def build(force=False, verbose=False):
    """Compile (if sources changed) and return the path of libpa.so."""
    os.makedirs(BUILD, exist_ok=True)
    stamp = os.path.join(BUILD, "digest")
    dig = _digest()
    if not force and os.path.exists(LIB) and os.path.exists(CALL) and os.path.exists(stamp):
        with open(stamp) as f:
            if f.read().strip() == dig:
                return LIB
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [nvcc] + ARCH + FLAGS + ["-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.append("-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s%s" % (src, r.stdout, r.stderr))
        if verbose:
            sys.stderr.write(r.stderr)
        return obj

    torch_dir, _ = _torch_dir()
    cuda_dir = os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))

    def compile_call():
        obj = os.path.join(BUILD, "pa_call.o")
        inc = [os.path.join(torch_dir, "include"),
               os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(cuda_dir, "include")]
        r = subprocess.run(["g++", "-O2", "-std=c++17", "-fPIC", "-c",
                            os.path.join(CSRC, "pa_call.cpp"), "-o", obj] + ["-I" + d for d in inc],
                           capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("g++ failed for pa_call.cpp:\n%s%s" % (r.stdout, r.stderr))
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        call = ex.submit(compile_call)
        objs = list(ex.map(compile_one, SOURCES))
        call = call.result()
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [nvcc] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB)
    tmp = CALL + ".tmp%d" % os.getpid()
    lib = os.path.join(torch_dir, "lib")
    r = subprocess.run(["g++", "-shared", "-o", tmp, call, "-L" + PKG, "-lpa", "-L" + lib,
                        "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
                        "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("linking _pa_call.so failed:\n%s%s" % (r.stdout, r.stderr))
    os.replace(tmp, CALL)
    with open(stamp, "w") as f:
        f.write(dig)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
