"""Build libfconv.so (the C-ABI library with its gfx950 kernels) and _call.so
(the Python module of csrc/call.cpp) in-tree.  _call.so is linked to torch and
left out where torch is not installed: nothing that needs it works there.

    python -m convolution_implicit_gemm_nhwc_amd.build

Kernels are compiled ahead of time for gfx950 only.  Flags:
  -ffp-contract=off   the int8 epilogue is specified operation by operation;
                      no multiply-add may be formed that the source does not
                      write (the side-input step calls fmaf explicitly);
  -fno-fast-math      IEEE semantics for the epilogues;
  -Xclang -target-feature -Xclang -packed-fp32-ops
                      no packed fp32 VALU instructions are generated.
"""
from __future__ import annotations

import importlib.util
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
INCLUDE = os.path.join(ROOT, "include")
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libfconv.so")
CALL = os.path.join(PKG, "_call.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

SOURCES = ["plan.cpp", "conv.hip", "wgrad.hip", "mx.hip", "xent.hip"]

COMMON = ["-O3", "-std=c++17", "-fPIC", "-ffp-contract=off", "-fno-fast-math",
          "-Wall", "-fvisibility=hidden", "-I", INCLUDE, "-I", CSRC]
DEVICE = ["--offload-arch=" + ARCH, "-Xclang", "-target-feature", "-Xclang",
          "-packed-fp32-ops"]


def build(verbose: bool = False) -> str:
    objs = []
    for src in SOURCES:
        path = os.path.join(CSRC, src)
        obj = os.path.join(CSRC, src + ".o")
        cmd = [HIPCC, *COMMON]
        if src.endswith(".hip"):
            cmd += DEVICE
        cmd += ["-c", path, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
        objs.append(obj)
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [HIPCC, "--offload-arch=" + ARCH, "-shared", "-fPIC", *objs, "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    for obj in objs:
        os.remove(obj)
    if importlib.util.find_spec("torch") is not None:
        build_call(verbose)
    else:
        if os.path.exists(CALL):  # of other sources
            os.remove(CALL)
        print("torch is not installed: %s not built (MxPlan, MxQuantPlan, XentPlan need it)" % CALL,
              file=sys.stderr, flush=True)
    return LIB


def build_call(verbose: bool = False) -> str:
    """The Python module of csrc/call.cpp, against the installed torch."""
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    tmp = CALL + ".tmp%d" % os.getpid()
    libs = os.path.join(root, "lib")
    cmd = [HIPCC, "-O2", "-std=c++17", "-fPIC", "-Wall", "-fvisibility=hidden", "-shared",
           "-no-hip-rt", "-DUSE_ROCM", "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI,
           "-I", INCLUDE, "-isystem", os.path.join(root, "include"),
           "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"], os.path.join(CSRC, "call.cpp"), "-o", tmp,
           "-L" + libs, "-lc10", "-lc10_hip", "-ltorch_cpu", "-ltorch_hip", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, CALL)
    return CALL


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
