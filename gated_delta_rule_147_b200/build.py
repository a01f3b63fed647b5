"""Builds the CUDA library in-tree: gated_delta_rule_147_b200/libgdr.so (sm_100a),
and, where torch is installed, the Python module of the layer operators beside
it, _layers.so.

Each source compiles to its own object (in parallel, under _build/), then one
link step each makes the shared library and the module (which links to it).

Usage: python -m gated_delta_rule_147_b200.build [--force] [--verbose]
"""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OBJDIR = os.path.join(ROOT, "_build")
SOURCES = ["api.cu", "decode.cu", "recurrent.cu", "chunk_sm100.cu", "chunk_erasefree_sm100.cu",
           "chunk_bwd.cu", "chunk_bwd_tc_sm100.cu", "chunk_bwd_grad_sm100.cu",
           "chunk_twopass_sm100.cu", "chunk_twopass256_sm100.cu", "chunk_twopass_general_sm100.cu", "selftest.cu",
           "static_scratch.cu", "conv.cu", "scan.cu", "scan_bwd.cu", "scan_api.cu", "qk_norm.cu"]
HEADERS = ["common.cuh", "chunk_common.cuh", "rcp_seed.h", "layer_common.cuh", "scan_common.cuh"]
BINDING = "layers_binding.cpp"
LIB = os.path.join(HERE, "libgdr.so")
MODULE = os.path.join(HERE, "_layers.so")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
COMPILE_FLAGS = [*ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                 "--expt-relaxed-constexpr"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "nvcc"


def _deps():
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS + [BINDING]]
    deps.append(os.path.join(ROOT, "include", "gdr.h"))
    return deps


def _torch_dir() -> str | None:
    """Where torch is installed (not imported: only its headers are wanted), or None:
    the library needs nvcc alone."""
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec and spec.origin else None


def _cuda_include() -> str:
    """The headers beside the nvcc in use."""
    nvcc = _nvcc()
    if not os.path.isabs(nvcc):
        nvcc = shutil.which(nvcc) or "/usr/local/cuda/bin/nvcc"
    return os.path.join(os.path.dirname(os.path.dirname(nvcc)), "include")


def _stale() -> bool:
    built = [LIB, MODULE] if _torch_dir() else [LIB]
    if not all(os.path.exists(f) for f in built):
        return True
    t = min(os.path.getmtime(f) for f in built)
    return any(os.path.getmtime(d) > t for d in _deps())


def _obj(src: str) -> str:
    return os.path.join(OBJDIR, os.path.splitext(src)[0] + ".o")


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        return LIB
    os.makedirs(OBJDIR, exist_ok=True)
    inc = ["-I", os.path.join(ROOT, "include")]
    # a header change rebuilds every object; otherwise only sources newer than their object
    hdr_t = max(os.path.getmtime(d) for d in _deps() if not d.endswith((".cu", ".cpp")))
    torch_dir = _torch_dir()
    cxx = os.environ.get("CXX", "g++")

    def compile_one(src: str):
        obj = _obj(src)
        path = os.path.join(CSRC, src)
        if not force and os.path.exists(obj) and os.path.getmtime(obj) > max(os.path.getmtime(path), hdr_t):
            return
        cmd = [_nvcc(), *COMPILE_FLAGS, *inc, "-c", "-o", obj, path]
        if src == BINDING:
            dirs = [os.path.join(torch_dir, "include"), os.path.join(torch_dir, "include/torch/csrc/api/include"),
                    sysconfig.get_paths()["include"], _cuda_include()]
            cmd = [cxx, "-O2", "-std=c++17", "-fPIC", *inc, *(f for d in dirs for f in ("-isystem", d)), "-c", "-o", obj,
                   path]
        if verbose:
            if src != BINDING:
                cmd.insert(1, "-Xptxas=-v")
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)

    with ThreadPoolExecutor(max_workers=min(len(SOURCES) + 1, os.cpu_count() or 4)) as ex:
        for f in [ex.submit(compile_one, s) for s in ([BINDING] if torch_dir else []) + SOURCES]:
            f.result()
    link = [_nvcc(), *ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", LIB, *[_obj(s) for s in SOURCES]]
    subprocess.run(link, check=True)
    if not torch_dir:
        return LIB
    libs = ["-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"]
    # by name, found beside the module: an absolute path would tie it to this folder
    subprocess.run([cxx, "-shared", "-o", MODULE, _obj(BINDING), "-L", HERE, "-l:libgdr.so", "-L",
                    os.path.join(torch_dir, "lib"), *libs,
                    "-Wl,-rpath,$ORIGIN"], check=True)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="--verbose" in sys.argv)
    print(LIB)
