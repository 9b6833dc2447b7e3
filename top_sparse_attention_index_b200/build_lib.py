"""Build libqsa.so (the C-ABI CUDA library) in-tree with nvcc for sm_100a, and _layer_ext.so
(the layer operators' torch-facing calls, host code only) with g++.

    python -m top_sparse_attention_index_b200.build_lib [--force] [--verbose-ptxas]

The library links the CUDA runtime statically, so the only run-time dependency is the
NVIDIA driver.  The extension links against the installed torch and libqsa.so beside it.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
from pathlib import Path

PKG = Path(__file__).resolve().parent
ROOT = PKG.parent
CSRC = PKG / "csrc"
INCLUDE = ROOT / "include"
LIBRARY = PKG / "libqsa.so"
EXTENSION = PKG / "_layer_ext.so"
EXT_SOURCE = CSRC / "qsa_torch.cpp"
SOURCES = [CSRC / "qsa_api.cu", CSRC / "qsa_attn.cu", CSRC / "qsa_noalloc.cu", CSRC / "qsa_probe.cu",
           CSRC / "qsa_probe_mma.cu", CSRC / "qsa_peer.cu",
           CSRC / "qsa_rope.cu", CSRC / "qsa_select.cu", CSRC / "qsa_decode.cu"]
DEPENDS = SOURCES + [CSRC / "qsa_layer.cuh", INCLUDE / "qsa_layer.h",
                     CSRC / "qsa_internal.h", CSRC / "qsa_ptx.cuh", INCLUDE / "qsa.h",
                     INCLUDE / "qsa_probe.h", INCLUDE / "qsa_peer.h"]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
    "--expt-relaxed-constexpr",
    "-Xcompiler", "-Wall",
]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and Path(cand).exists():
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libqsa.so")


def _stale(output: Path, depends) -> bool:
    return not output.exists() or output.stat().st_mtime < max(p.stat().st_mtime for p in depends)


def build_extension(force: bool = False) -> Path:
    """_layer_ext.so; libqsa.so has to be there."""
    if not force and not _stale(EXTENSION, [EXT_SOURCE, INCLUDE / "qsa_layer.h", INCLUDE / "qsa.h"]):
        return EXTENSION
    import torch
    root = Path(torch.__file__).resolve().parent
    cuda = Path(nvcc()).resolve().parent.parent
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", str(INCLUDE), "-isystem", str(root / "include"),
           "-isystem", str(root / "include/torch/csrc/api/include"),
           "-isystem", sysconfig.get_paths()["include"], "-isystem", str(cuda / "include"),
           str(EXT_SOURCE), "-o", str(EXTENSION), "-L", str(PKG), "-l:libqsa.so", "-Wl,-rpath,$ORIGIN",
           "-L", str(root / "lib"), "-ltorch_python", "-ltorch", "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    subprocess.run(cmd, check=True)
    return EXTENSION


def build(force: bool = False, verbose_ptxas: bool = False, output: Path = LIBRARY) -> Path:
    output = Path(output)
    if not force and not _stale(output, DEPENDS):
        if output == LIBRARY:
            build_extension()
        return output
    cmd = [nvcc(), *NVCC_FLAGS, "-I", str(INCLUDE), "-I", str(CSRC)]
    if verbose_ptxas:
        cmd += ["-Xptxas", "-v"]
    cmd += [str(s) for s in SOURCES] + ["-o", str(output)]
    subprocess.run(cmd, check=True)
    if output == LIBRARY:
        build_extension(force)
    return output


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="--verbose-ptxas" in sys.argv))
