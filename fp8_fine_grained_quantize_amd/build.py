"""Build libfp8blk.so (HIP, gfx950) in-tree with hipcc, and _layer_ext.so, the
C++ part of the Python binding, with the host compiler against torch.

    python -m fp8_fine_grained_quantize_amd.build
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libfp8blk.so")
EXT = os.path.join(PKG, "_layer_ext.so")
BUILD_DIR = os.path.join(PKG, "_build")

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CXX = os.environ.get("CXX", "g++")
ARCH = "gfx950"

COMMON_FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
    "-ffp-contract=off",                            # every FMA in the kernels is written explicitly
    "-fhip-fp32-correctly-rounded-divide-sqrt",     # fp32 '/' is IEEE round-to-nearest-even
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-mllvm", "-amdgpu-mfma-vgpr-form=1",           # MFMA results in VGPRs: the scale fold reads them with VALU
    "-Wno-unused-command-line-argument",
    f"-I{os.path.join(ROOT, 'include')}",
]

SOURCES = ["api.hip", "quantize.hip", "gemm.hip", "diag.hip", "moe.hip", "norm.hip", "grads.hip", "adamw.hip",
           "gated.hip"]
BINDING = ["layer_binding.cpp", "train_binding.cpp"]


def _run(what: str, cmd) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")


def _compile(src: str) -> str:
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    _run(f"hipcc for {src}", [HIPCC, *COMMON_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj])
    return obj


def _torch_dir() -> str:
    import torch
    return os.path.dirname(os.path.abspath(torch.__file__))


def _compile_binding(src: str) -> str:
    """A source of the binding's C++ part, against torch's headers (host code only)."""
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    inc = os.path.join(_torch_dir(), "include")
    _run(src, [CXX, "-std=c++17", "-O2", "-fPIC", "-fvisibility=hidden", f"-I{inc}",
                               f"-I{os.path.join(inc, 'torch', 'csrc', 'api', 'include')}",
                               f"-I{sysconfig.get_paths()['include']}", "-w", "-c",
                               os.path.join(CSRC, src), "-o", obj])
    return obj


def _link_binding(objs) -> None:
    lib = os.path.join(_torch_dir(), "lib")
    tmp = EXT + ".tmp"
    _run("link of the binding", [CXX, "-shared", "-o", tmp, *objs, f"-L{PKG}", "-l:libfp8blk.so", f"-L{lib}",
                                 "-ltorch_python", "-ltorch_cpu", "-lc10", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"])
    os.replace(tmp, EXT)


def build(verbose: bool = False) -> str:
    """Compile every HIP source for gfx950, link libfp8blk.so and the binding's
    C++ part; returns the library's path."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    srcs = [s for s in SOURCES if os.path.exists(os.path.join(CSRC, s))]
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs) + len(BINDING))) as ex:
        objs = ex.map(_compile, srcs)
        binding = list(ex.map(_compile_binding, BINDING))
        objs = list(objs)
    tmp = LIB + ".tmp"
    _run("link", [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs])
    os.replace(tmp, LIB)
    _link_binding(binding)
    if verbose:
        print(f"built {LIB}\nbuilt {EXT}")
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
