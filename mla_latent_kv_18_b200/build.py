"""Builds the sm_100a CUDA library ``libmla_b200.so`` in-tree with nvcc, and the
compiled binding ``_step.so`` of its packed-step calls with g++.

    python -m mla_latent_kv_18_b200.build [--force] [--verbose]

The library is a single translation unit (csrc/mla_api.cu includes every
kernel) exporting the C ABI of include/mla_decode.h and include/mla_step.h;
the binding (csrc/torch_step.cpp) links against it and torch.
"""
import importlib.metadata
import os
import shutil
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
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(shutil.which(NVCC) or NVCC)))
    return [CXX, "-O2", "-std=c++17", "-shared", "-fPIC",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            "-I", INCLUDE, "-I", os.path.join(at, "include"),
            "-I", os.path.join(at, "include", "torch", "csrc", "api", "include"),
            "-I", os.path.join(cuda, "include"), "-I", sysconfig.get_paths()["include"],
            os.path.join(CSRC, "torch_step.cpp"), "-o", out, "-L", PKG, "-l:libmla_b200.so", "-Wl,-rpath,$ORIGIN",
            "-L", os.path.join(at, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10",
            "-lc10_cuda"]


def _made_for():
    """What _step.so depends on besides its sources: it uses the C++ interfaces of torch and Python."""
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:   # a torch that no installer put there
        from torch import __version__ as version
    return f"torch {version}, {sys.implementation.cache_tag}"


def _made(out, sources, force, cmd, made_for=""):
    """Make `out` with cmd(path) if it is missing, older than a source, or made for something else
    (noted beside it)."""
    note = out + ".for"
    if not force and os.path.exists(out):
        t = os.path.getmtime(out)
        if all(os.path.getmtime(s) <= t for s in sources) and (not made_for or _read(note) == made_for):
            return
    tmp = out + ".tmp"
    subprocess.check_call(cmd(tmp))
    os.replace(tmp, out)
    if made_for:
        with open(note, "w") as f:
            f.write(made_for)


def _read(path):
    try:
        with open(path) as f:
            return f.read()
    except OSError:
        return ""


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the library and the binding where they are missing or older than their sources, the binding
    also where it was made for another torch or Python."""
    _made(LIB, _sources(), force, lambda out: nvcc_cmd(out, verbose))
    _made(STEP, _step_sources(), force, step_cmd, _made_for())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv))
