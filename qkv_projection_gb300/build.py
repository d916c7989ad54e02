"""Build libkaio_qkv.so in-tree with nvcc (sm_103a only).

Each .cu file is compiled to an object in parallel, then linked into one shared
library next to this file. The CUDA runtime is linked statically, so loading
the library needs no GPU; the driver is reached only at the first CUDA call.

_host.so, the Python module of host_calls.cpp, is compiled beside them against the
installed Python and torch. Where that cannot be done (no torch, no headers, no host
compiler) it is left out with a warning, and the calls that it shortens go through
Python; the library itself needs nvcc alone.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libkaio_qkv.so")
SOURCES = ["api.cu", "decode_w4a16.cu", "tc_decode.cu", "tc_kernels.cu", "dequant_group.cu",
           "rope.cu", "paged_decode.cu", "paged_chunk.cu"]
HOST_SOURCE = os.path.join(CSRC, "host_calls.cpp")
HOST_LIB = os.path.join(HERE, "_host.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found")
    return cand


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc(), *ARCH, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        cmd += ["-Xptxas", "-v"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{res.stdout}\n{res.stderr}")
    if verbose and res.stderr:
        sys.stderr.write(res.stderr)
    return obj


def _host_command(out: str):
    """The compiler's command for _host.so, or why there is none."""
    import sysconfig
    try:
        import torch
    except ImportError as e:
        return None, f"torch cannot be imported ({e})"
    include = sysconfig.get_paths()["include"]
    base = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    for needed in (os.path.join(include, "Python.h"), os.path.join(base, "include", "ATen", "ATen.h"),
                   os.path.join(base, "lib", "libc10_cuda.so")):
        if not os.path.exists(needed):
            return None, f"{needed} is missing"
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
            "-I", os.path.join(ROOT, "include"), "-isystem", include, "-isystem", cuda,
            "-isystem", os.path.join(base, "include"),
            "-isystem", os.path.join(base, "include", "torch", "csrc", "api", "include"),
            HOST_SOURCE, "-o", out, "-L", os.path.join(base, "lib"),
            "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"], ""


def _compile_host() -> None:
    """Builds _host.so, or says on stderr why it is left out; one of an earlier build goes."""
    tmp = HOST_LIB + ".tmp"
    cmd, why = _host_command(tmp)
    if cmd:
        try:
            res = subprocess.run(cmd, capture_output=True, text=True)
            if res.returncode == 0:
                os.replace(tmp, HOST_LIB)
                return
            why = f"g++ failed on {HOST_SOURCE}:\n{res.stdout}\n{res.stderr}"
        except OSError as e:
            why = f"g++ cannot be run ({e})"
    if os.path.exists(HOST_LIB):
        os.remove(HOST_LIB)
    sys.stderr.write(f"warning: built without {os.path.basename(HOST_LIB)}: {why}\n")


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        host = ex.submit(_compile_host)
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
        host.result()
    tmp = LIB + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
