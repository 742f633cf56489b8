"""When the CUDA library and the compiled binding are made again (nothing is compiled here)."""
import importlib.metadata
import os

import pytest

from mla_latent_kv_18_b200 import build as mla_build


@pytest.fixture
def made(tmp_path, monkeypatch):
    """build() with outputs in a folder of their own and a compiler that writes empty files: what it made."""
    out = []

    def compiler(cmd):
        path = cmd[cmd.index("-o") + 1]
        open(path, "w").close()
        out.append(os.path.basename(path).replace(".tmp", ""))

    monkeypatch.setattr(mla_build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(mla_build, "STEP", str(tmp_path / "_step.so"))
    monkeypatch.setattr(mla_build.subprocess, "check_call", compiler)

    def run(**kw):
        out.clear()
        mla_build.build(**kw)
        return list(out)
    return run


def test_made_once_and_by_force(made):
    assert made() == ["lib.so", "_step.so"]
    assert made() == []
    assert made(force=True) == ["lib.so", "_step.so"]


def test_the_binding_is_made_again_for_another_torch_or_python(made, monkeypatch):
    made()
    real = importlib.metadata.version
    monkeypatch.setattr(importlib.metadata, "version", lambda n: "9.9.0" if n == "torch" else real(n))
    assert made() == ["_step.so"]
    assert made() == []
    class Other:
        cache_tag = "cpython-999"
    monkeypatch.setattr(mla_build.sys, "implementation", Other)
    assert made() == ["_step.so"]
    assert made() == []


def test_older_than_a_source(made):
    made()
    os.utime(mla_build.STEP, (1, 1))
    assert made() == ["_step.so"]
    os.utime(mla_build.LIB, (1, 1))
    assert made() == ["lib.so"]


def test_nvcc_by_name(monkeypatch):
    """NVCC=nvcc on the path: the binding still finds CUDA's headers."""
    monkeypatch.setenv("PATH", os.path.dirname(mla_build.NVCC) + os.pathsep + os.environ["PATH"])
    monkeypatch.setattr(mla_build, "NVCC", "nvcc")
    cmd = mla_build.step_cmd("x.so")
    dirs = [cmd[i + 1] for i, a in enumerate(cmd) if a == "-I"]
    assert any(os.path.exists(os.path.join(d, "cuda_runtime_api.h")) for d in dirs), dirs
