"""Build libssd.so for sm_103a with nvcc (no cmake, no torch extension
machinery).  Each translation unit compiles in its own nvcc process, in
parallel, then one link step produces the shared library in-tree at
``state_space_model_chunked_gb300/_lib/libssd.so``.

Beside it, ``_lib/ssd_marshal.so`` is the Python module that hands tensors of
single-token calls to the library (compiled with the host compiler against torch's
headers, linked to libssd.so).

    python -m state_space_model_chunked_gb300.build [--force]
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_lib")
LIB = os.path.join(OUT_DIR, "libssd.so")
MARSHAL = os.path.join(OUT_DIR, "ssd_marshal.so")
OBJ_DIR = os.path.join(HERE, "_build")
SOURCES = ["api.cu", "decode.cu", "scan_simt.cu", "scan_tc.cu", "scan_static.cu", "widen.cu",
           "seqshard.cu", "api_layer.cu", "rmsnorm.cu", "gated_scan.cu", "linear_simt.cu",
           "linear_tc.cu", "linear_gemv.cu", "linear_few.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the SSD library needs the CUDA toolkit to build")
    return cand


def _flags():
    return ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                   "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def _compile_marshal() -> str:
    """The object file of marshal.cpp."""
    import torch
    from torch.utils import cpp_extension
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    inc = cpp_extension.include_paths() + [sysconfig.get_paths()["include"],
                                           os.path.join(cuda, "include"),
                                           os.path.join(ROOT, "include")]
    obj = os.path.join(OBJ_DIR, "marshal.o")
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    cmd = [os.environ.get("CXX") or shutil.which("g++") or "c++", "-O2", "-std=c++17", "-fPIC",
           f"-D_GLIBCXX_USE_CXX11_ABI={abi}", "-c", os.path.join(CSRC, "marshal.cpp"), "-o", obj]
    for d in inc:
        cmd += ["-isystem", d]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"host compiler failed on marshal.cpp:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_marshal(obj: str) -> None:
    from torch.utils import cpp_extension
    tmp = MARSHAL + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX") or shutil.which("g++") or "c++", "-shared", "-o", tmp, obj,
           "-L" + OUT_DIR, "-l:libssd.so", "-Wl,-rpath,$ORIGIN"]
    for d in cpp_extension.library_paths():
        cmd += ["-L" + d, "-Wl,-rpath," + d]
    cmd += ["-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of ssd_marshal.so failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, MARSHAL)


def _deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(ROOT, "include", "ssd.h"))
    return max(os.path.getmtime(f) for f in files)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every CUDA source for sm_103a and link libssd.so and ssd_marshal.so;
    returns libssd.so's path."""
    if not force and all(os.path.exists(f) and os.path.getmtime(f) >= _deps()
                         for f in (LIB, MARSHAL)):
        return LIB
    nvcc = _nvcc()
    os.makedirs(OUT_DIR, exist_ok=True)
    os.makedirs(OBJ_DIR, exist_ok=True)
    flags = _flags()

    def compile_one(src):
        obj = os.path.join(OBJ_DIR, src.replace(".cu", ".o"))
        cmd = [nvcc] + flags + ["-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd += ["-Xptxas", "-v"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and r.stderr:
            sys.stderr.write(r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        marshal = ex.submit(_compile_marshal)
        objs = list(ex.map(compile_one, SOURCES))
        marshal = marshal.result()
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    _link_marshal(marshal)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
