"""Build libiqcodec.so and its Python binding in-tree with hipcc for gfx950.

Every HIP source under csrc/ is compiled for gfx950 only, without packed-FP32
instructions and without floating-point contraction (the encode's keys are
recomputed bit-for-bit during index recovery), and linked into one shared
library that exports the C-ABI of include/iq_codec.h and include/iq_layers.h.
csrc/binding.cpp, host code only, becomes the extension module of the layer
operators' binding.
"""

from __future__ import annotations

import glob
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libiqcodec.so")
BINDING = os.path.join(PKG, "_layers.so")
BUILD_DIR = os.path.join(PKG, "_build")

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-ffp-contract=off",
    "-fno-fast-math",
    "-mcode-object-version=5",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", INCLUDE,
    "-I", CSRC,
    "-Wall",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.hip")))


def build(verbose: bool = False) -> str:
    """Compile every csrc/*.hip and link libiqcodec.so; returns its path."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    objs = []
    for src in sources():
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-4] + ".o")
        cmd = [HIPCC, *FLAGS, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        # hipcc's host pass does not know the packed-fp32 target feature and
        # says so; that note is harmless and filtered out.
        noise = "is not a recognized feature for this target"
        msg = "\n".join(l for l in (r.stdout + r.stderr).splitlines() if noise not in l)
        if r.returncode != 0:
            raise RuntimeError("hipcc failed for %s:\n%s" % (src, msg))
        if msg.strip() and verbose:
            print(msg, file=sys.stderr)
        objs.append(obj)
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", tmp,
           "-Wl,-rpath,/opt/rocm/lib"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s" % (r.stdout + r.stderr))
    os.replace(tmp, LIB)
    build_binding(verbose)
    return LIB


def build_binding(verbose: bool = False) -> str:
    """Compile csrc/binding.cpp against PyTorch's headers; returns its path.  The
    libraries of PyTorch that it names are those that ``import torch`` has loaded."""
    from torch.utils.cpp_extension import include_paths, library_paths
    tmp = BINDING + ".tmp%d" % os.getpid()
    # As plain C++, where hipcc adds neither HIP's headers nor its platform.
    rocm = os.path.dirname(os.path.dirname(os.path.realpath(HIPCC)))
    cmd = [HIPCC, "-x", "c++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           "-D__HIP_PLATFORM_AMD__"]
    for path in [*include_paths(), sysconfig.get_paths()["include"], os.path.join(rocm, "include")]:
        cmd += ["-isystem", path]
    cmd += ["-I", INCLUDE, os.path.join(CSRC, "binding.cpp"), "-o", tmp, "-L", PKG, "-liqcodec",
            "-Wl,-rpath,$ORIGIN"]
    for path in library_paths():
        cmd += ["-L", path]
    cmd += ["-ltorch_python", "-ltorch_cpu", "-lc10_hip", "-lc10"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("hipcc failed for binding.cpp:\n%s" % (r.stdout + r.stderr))
    os.replace(tmp, BINDING)
    return BINDING


if __name__ == "__main__":
    print(build(verbose=True))
