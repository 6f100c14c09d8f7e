"""Build libw4a4.so (hipcc, gfx950) and the native binding _native.so (g++,
host code only; needs PyTorch's headers) in-tree.

    python -m hadamard_rotated_w4a4_amd.build
"""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libw4a4.so")
CEILINGS_LIB = os.path.join(PKG, "libw4a4_ceilings.so")  # measured ceilings for the benchmark
NATIVE = os.path.join(PKG, "_native.so")  # the binding's native part
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CXX = os.environ.get("CXX", "g++")  # the native binding's host compiler

SOURCES = [os.path.join(CSRC, f) for f in ("w4a4.hip", "rows.hip", "mx4.hip", "kv.hip")]
HEADERS = [os.path.join(CSRC, h) for h in ("abi.h", "common.h", "k_prep.h", "k_rotq.h", "k_route.h", "k_dense.h", "k_smallm.h", "k_grouped.h", "k_w16.h",
                                            "k_rows.h", "k_mx4.h", "k_kv.h", "k_attend.h")] + [
    os.path.join(ROOT, "include", "w4a4.h")]

FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-shared",
    # no packed-FP32 instructions anywhere in the device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # no silent multiply-add fusion: the quantisers' codes depend on every
    # rounding step; the GEMM epilogue asks for its fused multiply-adds by name
    "-ffp-contract=off",
    # matrix-core results straight into VGPRs: no accvgpr reads in the epilogue
    "-mllvm", "-amdgpu-mfma-vgpr-form",
    "-Wall",
    "-Wno-unused-command-line-argument",
]


def build(verbose: bool = False) -> str:
    """Compile the HIP sources into libw4a4.so and the ceiling probes into
    libw4a4_ceilings.so, then the native binding (always recompiles).  The C
    libraries need hipcc only: without PyTorch and its headers they are built
    and the binding is left out, with a note."""
    _compile(LIB, SOURCES, verbose)
    _compile(CEILINGS_LIB, [os.path.join(CSRC, "ceilings.hip")], verbose)
    home = _pytorch()
    if home is None:
        print("PyTorch's headers not found: libw4a4.so is built, the Python binding's _native.so is not", flush=True)
    else:
        _compile_native(home, verbose)
    return LIB


def _pytorch():
    """The folder of the PyTorch package with its headers, or None."""
    spec = importlib.util.find_spec("torch")
    home = os.path.dirname(spec.origin) if spec and spec.origin else None
    header = home and os.path.join(home, "include", "torch", "csrc", "autograd", "python_variable.h")
    return home if header and os.path.exists(header) else None


def _rocm_include() -> str:
    """The HIP headers of the ROCm that HIPCC belongs to."""
    path = shutil.which(HIPCC) or HIPCC
    for hipcc in (path, os.path.realpath(path)):  # <rocm>/bin/hipcc, itself or behind a link
        include = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(hipcc))), "include")
        if os.path.exists(os.path.join(include, "hip", "hip_runtime.h")):
            return include
    raise RuntimeError(f"no HIP headers beside {HIPCC}")


def _compile_native(home: str, verbose: bool) -> None:
    """csrc/binding.cpp against the headers of PyTorch at `home` and libw4a4.so."""
    includes = [os.path.join(home, "include"), os.path.join(home, "include", "torch", "csrc", "api", "include"),
                sysconfig.get_paths()["include"], _rocm_include(), os.path.join(ROOT, "include")]
    libs = os.path.join(home, "lib")
    tmp = NATIVE + ".tmp"
    cmd = [CXX, "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
           *(f"-isystem{i}" for i in includes), "-o", tmp, os.path.join(CSRC, "binding.cpp"), f"-L{PKG}", "-l:" + os.path.basename(LIB),
           f"-L{libs}", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_hip", "-lc10", "-lc10_hip", f"-Wl,-rpath,$ORIGIN:{libs}"]
    _run(cmd, CXX, verbose)
    os.replace(tmp, NATIVE)


def _run(cmd: list, tool: str, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    # the host pass does not know the packed-fp32 feature; that note is harmless
    noise = "is not a recognized feature for this target"
    out = "\n".join(ln for ln in (res.stdout + res.stderr).splitlines() if noise not in ln)
    if res.returncode != 0:
        raise RuntimeError(f"{tool} failed ({res.returncode}):\n{out}")
    if verbose and out.strip():
        print(out)


def _compile(lib: str, sources: list, verbose: bool) -> None:
    tmp = lib + ".tmp"
    cmd = [HIPCC, *FLAGS, "-I", os.path.join(ROOT, "include"), "-o", tmp, *sources]
    _run(cmd, "hipcc", verbose)
    os.replace(tmp, lib)


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
