"""Build the CUDA library (sm_100a) in-tree: bit_quantized_linear_svdq_b200/_lib/libsvdq_b200.so, and the Python
extension module beside it that calls it with torch tensors (_lib/_attn_torch.so).

Usage:  python -m bit_quantized_linear_svdq_b200.build [--verbose]

Compiles every csrc/*.cu with nvcc for sm_100a only (the kernels use tcgen05,
TMA and the FP4 converts, which exist on that target alone) and links one
shared library exporting the C ABI declared in include/svdq.h and
include/svdq_attn.h.
"""
from __future__ import annotations

import glob
import hashlib
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIBDIR = os.path.join(PKG, "_lib")
LIB = os.path.join(LIBDIR, "libsvdq_b200.so")
EXT = os.path.join(LIBDIR, "_attn_torch.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "--expt-relaxed-constexpr",
]


CXX_FLAGS = ["-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden"]


def _torch_version() -> str:
    from torch.version import __version__
    return __version__


def _cxx() -> str:
    for cand in (os.environ.get("CXX"), shutil.which("g++"), shutil.which("c++")):
        if cand and (os.path.exists(cand) or shutil.which(cand)):
            return cand
    raise RuntimeError("no C++ compiler found")


def _extension_commands(obj: str, cuda: str):
    """Commands that compile csrc/attn_torch.cpp to `obj`, and link it beside the library."""
    import torch
    base = os.path.dirname(torch.__file__)
    inc = [os.path.join(ROOT, "include"), os.path.join(base, "include"),
           os.path.join(base, "include", "torch", "csrc", "api", "include"), os.path.join(cuda, "include"),
           sysconfig.get_paths()["include"]]
    abi = f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"
    comp = [_cxx(), *CXX_FLAGS, abi, *[f"-I{i}" for i in inc], "-c", os.path.join(CSRC, "attn_torch.cpp"), "-o", obj]
    link = [_cxx(), "-shared", "-o", EXT + ".tmp", obj, f"-L{LIBDIR}", "-l:libsvdq_b200.so", "-Wl,-rpath,$ORIGIN",
            f"-L{os.path.join(base, 'lib')}", "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    return comp, link


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    deps = srcs + sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) +
                         glob.glob(os.path.join(CSRC, "*.cpp")))
    deps += sorted(glob.glob(os.path.join(ROOT, "include", "*.h")))
    return srcs, deps


def _digest(deps) -> str:
    h = hashlib.sha256()
    h.update(" ".join(NVCC_FLAGS).encode())
    h.update(" ".join([sys.version, _torch_version(), *CXX_FLAGS]).encode())    # the extension module's ABI
    for d in deps:
        with open(d, "rb") as f:
            # Paths relative to the repository: a copy of the tree elsewhere
            # (with its built library) keeps the same digest.
            h.update(os.path.relpath(d, ROOT).encode())
            h.update(f.read())
    return h.hexdigest()


def build(verbose: bool = False, force: bool = False) -> str:
    srcs, deps = _sources()
    stamp = LIB + ".sha256"
    digest = _digest(deps)
    if not force and os.path.exists(LIB) and os.path.exists(EXT) and os.path.exists(stamp):
        with open(stamp) as f:
            if f.read().strip() == digest:
                return LIB
    os.makedirs(LIBDIR, exist_ok=True)
    objdir = os.path.join(LIBDIR, "obj")
    os.makedirs(objdir, exist_ok=True)
    nvcc = _nvcc()
    objs, cmds = [], []
    for src in srcs:
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        cmd = [nvcc, *NVCC_FLAGS, "-I", os.path.join(ROOT, "include"), "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
            print(" ".join(cmd), flush=True)
        cmds.append(cmd)
        objs.append(obj)
    ext_obj = os.path.join(objdir, "attn_torch.cpp.o")
    compile_ext, link_ext = _extension_commands(ext_obj, os.path.dirname(os.path.dirname(os.path.realpath(nvcc))))
    cmds.append(compile_ext)
    # One compiler process per source, as many at once as there are cores.
    from concurrent.futures import ThreadPoolExecutor
    with ThreadPoolExecutor(max_workers=max(1, min(len(cmds), os.cpu_count() or 1))) as pool:
        for r in list(pool.map(lambda c: subprocess.run(c, capture_output=not verbose, text=True), cmds)):
            if r.returncode != 0:
                raise RuntimeError("compiling failed: " + " ".join(r.args) + "\n" + (r.stderr or "") + (r.stdout or ""))
    tmp = LIB + ".tmp"
    cmd = [nvcc, "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-o", tmp, *objs, "-lcudart_static",
           "-Xcompiler", "-fvisibility=hidden"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    subprocess.run(link_ext, check=True)
    os.replace(EXT + ".tmp", EXT)
    with open(stamp, "w") as f:
        f.write(digest)
    return LIB


if __name__ == "__main__":
    print(build(verbose="--verbose" in sys.argv, force="--force" in sys.argv))
