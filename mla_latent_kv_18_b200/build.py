"""Builds the sm_100a CUDA library ``libmla_b200.so`` in-tree with nvcc, and the
compiled binding ``_step.so`` of its packed-step calls with g++.

    python -m mla_latent_kv_18_b200.build [--force] [--verbose]

The library is a single translation unit (csrc/mla_api.cu includes every
kernel) exporting the C ABI of include/mla_decode.h and include/mla_step.h;
the binding (csrc/torch_step.cpp) links against it and torch.
"""
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libmla_b200.so")
STEP = os.path.join(PKG, "_step.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
CXX = os.environ.get("CXX", "g++")


def _headers():
    return [os.path.join(INCLUDE, f) for f in sorted(os.listdir(INCLUDE)) if f.endswith(".h")]


def _sources():
    out = _headers()
    for f in sorted(os.listdir(CSRC)):
        if f.endswith((".cu", ".cuh", ".h")):
            out.append(os.path.join(CSRC, f))
    return out


def _step_sources():
    return _headers() + [os.path.join(CSRC, "torch_step.cpp")]


def nvcc_cmd(out=LIB, verbose=False):
    cmd = [NVCC, "-O3", "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo",
           "--use_fast_math", "-Xcompiler", "-fPIC", "-shared", "-I", INCLUDE, "-I", CSRC,
           "-o", out, os.path.join(CSRC, "mla_api.cu")]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    return cmd


def step_cmd(out=STEP):
    import torch
    at = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(NVCC))
    return [CXX, "-O2", "-std=c++17", "-shared", "-fPIC",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            "-I", INCLUDE, "-I", os.path.join(at, "include"),
            "-I", os.path.join(at, "include", "torch", "csrc", "api", "include"),
            "-I", os.path.join(cuda, "include"), "-I", sysconfig.get_paths()["include"],
            os.path.join(CSRC, "torch_step.cpp"), "-o", out, "-L", PKG, "-l:libmla_b200.so", "-Wl,-rpath,$ORIGIN",
            "-L", os.path.join(at, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10",
            "-lc10_cuda"]


def _made(out, sources, force, cmd):
    """Make `out` with cmd(path) if it is missing or older than a source."""
    if not force and os.path.exists(out):
        t = os.path.getmtime(out)
        if all(os.path.getmtime(s) <= t for s in sources):
            return
    tmp = out + ".tmp"
    subprocess.check_call(cmd(tmp))
    os.replace(tmp, out)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the library and the binding where they are missing or older than their sources."""
    _made(LIB, _sources(), force, lambda out: nvcc_cmd(out, verbose))
    _made(STEP, _step_sources(), force, step_cmd)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv))
