"""Build the HIP library fp32_gemm_nn_amd/libmisgemm.so for gfx950.

The tensor forms' binding (_binding.so) is host code, compiled against torch's
headers. hipcc cross-compiles the device code without a GPU present. Packed-FP32 VALU
instructions are switched off for all device code. The sources are compiled
to objects in parallel (under fp32_gemm_nn_amd/_build/) and linked into one
shared library.
"""
from __future__ import annotations

import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SRCS = [os.path.join(PKG, "csrc", name) for name in ("misgemm.hip", "ladder.hip", "scratch.hip", "clock_probe.hip",
                                                "fp8_gemm.hip", "fp8_direct.hip", "fp8_tile.hip",
                                                "fp8_quantize.hip", "rmsnorm.hip")]
OBJ_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmisgemm.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
    "-Wall", "-Wno-unused-function",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"),
]


BINDING_SRC = os.path.join(PKG, "csrc", "binding.cpp")
BINDING = os.path.join(PKG, "_binding.so")
CXX = os.environ.get("CXX", "g++")


def binding_command(out: str) -> list[str]:
    import sysconfig

    import torch

    home = os.path.dirname(torch.__file__)
    libs = os.path.join(home, "lib")
    return [CXX, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            "-isystem", os.path.join(home, "include"),
            "-isystem", os.path.join(home, "include", "torch", "csrc", "api", "include"),
            "-isystem", sysconfig.get_paths()["include"],
            BINDING_SRC, "-o", out, "-L" + libs, "-ltorch_python", "-ltorch_cpu", "-lc10"]


def build(verbose: bool = False, extra: list[str] | None = None) -> str:
    os.makedirs(OBJ_DIR, exist_ok=True)
    procs = []
    objs = []
    for src in SRCS:
        obj = os.path.join(OBJ_DIR, os.path.splitext(os.path.basename(src))[0] + ".o")
        cmd = [HIPCC, *FLAGS, *(extra or []), "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((cmd, subprocess.Popen(cmd)))
        objs.append(obj)
    # The tensor forms' binding is for torch: without it the library alone is
    # built, and a binding of an earlier one does not stay beside it.
    try:
        binding = binding_command(BINDING + ".tmp")
    except ModuleNotFoundError as e:
        if e.name != "torch":
            raise
        binding = None
        print("no torch: the library alone, without the tensor forms' binding", file=sys.stderr)
    if binding is not None:
        if verbose:
            print(" ".join(binding), flush=True)
        procs.append((binding, subprocess.Popen(binding)))
    for cmd, p in procs:
        if p.wait() != 0:
            raise subprocess.CalledProcessError(p.returncode, cmd)
    link = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", LIB + ".tmp"]
    if verbose:
        print(" ".join(link), flush=True)
    subprocess.run(link, check=True)
    os.replace(LIB + ".tmp", LIB)
    if binding is not None:
        os.replace(BINDING + ".tmp", BINDING)
    elif os.path.exists(BINDING):
        os.remove(BINDING)
    return LIB


if __name__ == "__main__":
    extra = [a for a in sys.argv[1:] if a != "-v"]
    print(build(verbose="-v" in sys.argv, extra=extra))
