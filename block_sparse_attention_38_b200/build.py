"""Build the C-ABI shared library libbsa.so in-tree with nvcc for sm_100a, and the
binding's marshalling module _bsa_torch.so with g++ against torch's headers.

    python -m block_sparse_attention_38_b200.build [--force] [--verbose-ptxas]

The library holds the host pattern builder (bsa_pattern.cpp) and the CUDA
translation units: the forward launcher with its kernel (bsa_forward.cu),
top-k block selection (bsa_topk.cu), the decode step (bsa_decode.cu), the
backward pass (bsa_backward.cu), the 4-bit cache (bsa_q4_cache.cu) and the
decode steps over long caches (bsa_stream_decode.cu) and sliding-window
attention (bsa_window_fwd.cu, bsa_window_bwd.cu).  CUDA runtime is linked
statically; the driver's tensor-map encoder is looked up at run time, so the
library loads on a machine without a GPU (only compute calls need one).
"""
from __future__ import annotations

import argparse
import importlib.util
import os
import runpy
import subprocess
import sys
import sysconfig

from .long_stream import marshal_tag

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
SOURCES = [os.path.join(CSRC, "bsa_pattern.cpp"), os.path.join(CSRC, "bsa_forward.cu"),
           os.path.join(CSRC, "bsa_topk.cu"), os.path.join(CSRC, "bsa_decode.cu"),
           os.path.join(CSRC, "bsa_backward.cu"), os.path.join(CSRC, "bsa_q4_cache.cu"),
           os.path.join(CSRC, "bsa_stream_decode.cu"), os.path.join(CSRC, "bsa_window_fwd.cu"),
           os.path.join(CSRC, "bsa_window_bwd.cu")]
DEPS = SOURCES + [os.path.join(CSRC, f) for f in sorted(os.listdir(CSRC)) if f.endswith(".cuh")] + [
    os.path.join(ROOT, "include", "bsa.h")]
LIB = os.path.join(HERE, "libbsa.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "--threads", "0", "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
    "--expt-relaxed-constexpr",
    "-I" + os.path.join(ROOT, "include"),
]


MARSHAL_SOURCE = os.path.join(CSRC, "bsa_torch.cpp")
MARSHAL = os.path.join(HERE, "_bsa_torch.so")


def stale(target=LIB, deps=None) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(p) > t for p in (DEPS if deps is None else deps))


def torch_home():
    """Folder and version of the torch that this Python would import, without importing
    it; (None, None) where there is none."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return None, None
    at = spec.submodule_search_locations[0]
    return at, str(runpy.run_path(os.path.join(at, "version.py"))["__version__"])


def marshal_stale(version: str) -> bool:
    """Whether sources are newer than the module, or its file does not hold the text that
    says what it was built for."""
    if stale(MARSHAL, [MARSHAL_SOURCE, os.path.join(ROOT, "include", "bsa.h")]):
        return True
    with open(MARSHAL, "rb") as f:
        return marshal_tag(version).encode() not in f.read()


def build_marshal(force: bool = False):
    """_bsa_torch.so, for the torch and Python at hand; None where there is no torch,
    without which only the calls that take tensors are missing."""
    at, version = torch_home()
    if at is None:
        print("no torch: _bsa_torch.so is not built", file=sys.stderr)
        return None
    if not force and not marshal_stale(version):
        return MARSHAL
    cuda = os.path.dirname(os.path.dirname(NVCC))
    tmp = MARSHAL + f".tmp{os.getpid()}"
    subprocess.run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
                    f'-DBSA_BUILT_FOR="{marshal_tag(version)}"',
                    "-I" + os.path.join(ROOT, "include"), "-I" + os.path.join(at, "include"),
                    "-I" + sysconfig.get_paths()["include"], "-I" + os.path.join(cuda, "include"), MARSHAL_SOURCE,
                    "-o", tmp, "-L" + os.path.join(at, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10",
                    "-lc10_cuda"], check=True)
    os.replace(tmp, MARSHAL)
    return MARSHAL


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """The library, which needs nvcc only, and then the binding's module."""
    if force or stale():
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [NVCC] + FLAGS + (["-Xptxas", "-v"] if verbose_ptxas else []) + SOURCES + ["-o", tmp]
        subprocess.run(cmd, check=True)
        os.replace(tmp, LIB)
    build_marshal(force)
    return LIB


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose-ptxas", action="store_true")
    args = ap.parse_args(argv)
    print(build(force=args.force, verbose_ptxas=args.verbose_ptxas))


if __name__ == "__main__":
    sys.exit(main())
