"""Build the HIP libraries (libvrc.so, libvrc_ops.so) for gfx950 with hipcc, in-tree,
and the compiled Python binding of the model's operators (_vrc_model.so) with g++."""
from __future__ import annotations

import importlib.util
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
CSRC_OPS = os.path.join(PKG, "csrc_ops")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libvrc.so")
LIB_OPS = os.path.join(PKG, "libvrc_ops.so")
# One translation unit per element type holds that type's kernels; vrc_api.hip
# holds the C ABI.  They compile in parallel.
SOURCES = [os.path.join(CSRC, f) for f in
           ("vrc_type_bf16.hip", "vrc_type_f16.hip", "vrc_type_f32.hip", "vrc_type_i32.hip", "vrc_api.hip")]
# The tensor-parallel layer's and model's operators (include/vrc_ops.h, vrc_model.h) are a library of
# their own: libvrc.so's kernels only stream through registers, and its tests
# pin that; these use LDS and the matrix cores.  They have a directory of their own
# as well: the recorded counters of libvrc.so's kernels are tied to the bytes of csrc/.
SOURCES_OPS = [os.path.join(CSRC_OPS, f) for f in
               ("vrc_mx4_matmul.hip", "vrc_dropout.hip", "vrc_mx4.hip", "vrc_ops_api.hip", "vrc_cross_entropy_f32.hip",
                "vrc_cross_entropy_f16.hip", "vrc_cross_entropy_bf16.hip", "vrc_layer_norm.hip", "vrc_model_api.hip")]
OBJDIR = os.path.join(PKG, "_build")

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-fvisibility=hidden",
    # Adds only, but never let the compiler contract or reassociate them.
    "-ffp-contract=off",
    "-fno-fast-math",
    "-fno-gpu-flush-denormals-to-zero",
    # Keep packed-fp32 instructions out of the generated code.
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall",
    "-Wno-unused-command-line-argument",
]


C_CHECK_SRC = os.path.join(ROOT, "tests", "c", "vrc_c_check.c")
C_CHECK_BIN = os.path.join(ROOT, "tests", "c", "vrc_c_check")


def build_c_check(verbose: bool = False) -> str:
    """Build the plain-C user of the ABI (tests/c/vrc_c_check.c) against
    libvrc.so and /opt/rocm's HIP runtime."""
    cmd = ["gcc", "-O2", "-std=c11", "-Wall", "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include", "-I", INCLUDE,
           "-o", C_CHECK_BIN, C_CHECK_SRC, "-L", PKG, "-lvrc", "-L", "/opt/rocm/lib", "-lamdhip64",
           "-Wl,-rpath,$ORIGIN/../../ring_all_reduce_virtual_amd", "-Wl,-rpath,/opt/rocm/lib"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    return C_CHECK_BIN


CVT_CHECK_SRC = os.path.join(ROOT, "tests", "c", "bf16_cvt_check.hip")
CVT_CHECK_BIN = os.path.join(ROOT, "tests", "c", "bf16_cvt_check")


def build_cvt_check(verbose: bool = False) -> str:
    """Build the exhaustive check of the bf16 conversion the kernels use
    (tests/c/bf16_cvt_check.hip), with the library's compiler flags."""
    flags = [f for f in FLAGS if f not in ("-fPIC", "-fvisibility=hidden")]
    cmd = [HIPCC, *flags, "-o", CVT_CHECK_BIN, CVT_CHECK_SRC]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    return CVT_CHECK_BIN


BINDING_SRC = os.path.join(CSRC_OPS, "vrc_model_binding.cpp")
BINDING_LIB = os.path.join(PKG, "_vrc_model.so")


def build_binding(verbose: bool = False) -> str | None:
    """Build the compiled Python binding of include/vrc_model.h against torch's
    headers and libvrc_ops.so (host code only).  Without torch, whose tensors it takes,
    there is none: the libraries serve callers of their C ABI."""
    import sysconfig

    spec = importlib.util.find_spec("torch")
    if spec is None:
        print("torch is not installed: the model operators' Python binding is not built", flush=True)
        return None
    torch = os.path.dirname(spec.origin)
    tmp = BINDING_LIB + ".tmp"
    system = [os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
              sysconfig.get_paths()["include"], "/opt/rocm/include"]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall", "-Wno-attributes", "-DUSE_ROCM",
           "-D__HIP_PLATFORM_AMD__=1", *(a for d in system for a in ("-isystem", d)), "-I", INCLUDE, "-o", tmp, BINDING_SRC,
           "-L", PKG, "-l:libvrc_ops.so", "-L", os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10",
           "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, BINDING_LIB)
    return BINDING_LIB


def build(verbose: bool = False, jobs: int = 0) -> str:
    """Compile every source to an object (in parallel), link libvrc.so and
    libvrc_ops.so and the binding on it, and return libvrc.so's path."""
    os.makedirs(OBJDIR, exist_ok=True)
    sources = SOURCES + SOURCES_OPS
    jobs = jobs or min(len(sources), os.cpu_count() or 1, 16)
    objs, pending = {}, []
    for src in sources:
        obj = os.path.join(OBJDIR, os.path.basename(src) + ".o")
        objs[src] = obj
        cmd = [HIPCC, *FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", "-o", obj, src]
        if verbose:
            print(" ".join(cmd), flush=True)
        pending.append(cmd)
    running = []
    failed = None
    while pending or running:
        while pending and len(running) < jobs:
            cmd = pending.pop(0)
            running.append((cmd, subprocess.Popen(cmd)))
        cmd, proc = running.pop(0)
        if proc.wait() != 0 and failed is None:
            failed = cmd
    if failed is not None:
        raise subprocess.CalledProcessError(1, failed)
    for lib, srcs in ((LIB, SOURCES), (LIB_OPS, SOURCES_OPS)):
        tmp = lib + ".tmp"
        cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp, *(objs[s] for s in srcs)]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
        os.replace(tmp, lib)
    build_binding(verbose)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    build_c_check(verbose=True)
    build_cvt_check(verbose=True)
    sys.exit(0)
