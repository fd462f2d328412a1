"""Build libpa.so in-tree with nvcc for sm_103a, and the Python marshalling module _marshal.

Each source is compiled to an object in parallel (one -gencode, -lineinfo), then
linked into ``paged_kv_cache_126_gb300/libpa.so``; ``csrc/marshal.cpp`` becomes
``paged_kv_cache_126_gb300/_marshal.so`` beside it.  A rebuild happens only when a
source or header is newer than the libraries, or torch is another than _marshal was built against.
"""

from __future__ import annotations

import concurrent.futures as cf
import importlib.metadata
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libpa.so")
MARSHAL = os.path.join(PKG, "_marshal.so")
MARSHAL_TORCH = os.path.join(BUILD, "_marshal.torch")  # the torch version that _marshal.so was built against

SOURCES = ["block_manager.cpp", "api.cu", "append.cu", "decode_f16.cu", "decode_bf16.cu", "decode_f32.cu",
           "prefill.cu", "decode_split.cu", "decode_shared.cu", "rotary.cu", "decode_q4.cu", "decode_selected.cu",
           "select.cu"]
GENCODE = "-gencode=arch=compute_103a,code=sm_103a"


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpa")


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "pa.h"))
    files.append(os.path.abspath(__file__))
    return files


def _torch_version() -> str:
    try:
        return importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        import torch

        return torch.__version__


def is_stale() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(MARSHAL) or not os.path.exists(MARSHAL_TORCH):
        return True
    with open(MARSHAL_TORCH) as f:
        if f.read() != _torch_version():
            return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(MARSHAL))
    return any(os.path.getmtime(f) > t for f in _inputs())


def _compile(nvcc: str, src: str, extra) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc, GENCODE, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
           "-I", INCLUDE, "-I", CSRC, "-c", os.path.join(CSRC, src), "-o", obj] + list(extra)
    if src.endswith(".cu"):
        cmd += ["-Xptxas", "-warn-spills"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{res.stdout}\n{res.stderr}")
    if res.stderr.strip():
        sys.stderr.write(res.stderr)
    return obj


def _build_marshal() -> str:
    """The extension module _marshal (host code against torch's headers; no CUDA code)."""
    import sysconfig

    import torch

    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    include = [INCLUDE, os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    tmp = MARSHAL + f".tmp{os.getpid()}"
    cmd = [shutil.which("g++") or "g++", "-std=c++17", "-O2", "-fPIC", "-shared", "-w",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    cmd += [f"-I{d}" for d in include]
    cmd += [os.path.join(CSRC, "marshal.cpp"), "-o", tmp, f"-L{os.path.join(root, 'lib')}", "-lc10", "-lc10_cuda", "-ltorch_cpu",
            "-ltorch_python"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed for marshal.cpp:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, MARSHAL)
    with open(MARSHAL_TORCH, "w") as f:
        f.write(_torch_version())
    return MARSHAL


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    """Compile every CUDA/C++ source of libpa and link the shared library."""
    if not force and not is_stale():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(len(SOURCES) + 1, os.cpu_count() or 4)) as ex:
        marshal = ex.submit(_build_marshal)
        objs = list(ex.map(lambda s: _compile(nvcc, s, extra), SOURCES))
        marshal.result()
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, GENCODE, "-shared", "-o", tmp] + objs
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
