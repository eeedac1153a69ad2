"""The CUDA context that calls work in, without a GPU: csrc/handle.h compiled
against a model of current contexts (tests/c_abi/context_check.cpp)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("no g++")
    out = str(tmp_path_factory.mktemp("context") / "context_check")
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    r = subprocess.run(["g++", "-std=c++17", "-Wall", "-O1", "-I",
                        os.path.join(ROOT, "dense_gemm_sm100_gb300", "csrc"), "-isystem", os.path.join(cuda, "include"),
                        os.path.join(ROOT, "tests", "c_abi", "context_check.cpp"), "-o", out],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return out


@pytest.mark.parametrize("scenario", ["same", "other", "none", "making"])
def test_context(program, scenario):
    r = subprocess.run([program, scenario], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout + r.stderr
