"""The orthogonalised update's entry points without a GPU."""
import ctypes
import math
import os
import re
import shutil
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gemm_ortho.h")
P = 0x10000  # a fake, aligned address: the checks never dereference


@pytest.fixture(scope="module")
def g():
    from dense_gemm_sm100_gb300 import build, gemm
    build.build()
    gemm.load_library()
    return gemm


def test_declared_functions_are_exported_and_bound(g):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(gemm_[a-z0-9_]+)\s*\(", text))
    assert len(names) == 2
    for n in names:
        assert hasattr(g.load_library(), n) and hasattr(g, n), n
    assert g.GEMM_ORTHO_MAX_STEPS == int(re.search(r"GEMM_ORTHO_MAX_STEPS (\d+)", text).group(1))


def test_header_is_plain_c(tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("no gcc")
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    src = tmp_path / "use.c"
    src.write_text('#include "gemm_ortho.h"\nint main(void) { return GEMM_ORTHO_MAX_STEPS > 0 ? 0 : 1; }\n')
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"),
                        "-isystem", os.path.join(cuda, "include"), "-c", str(src), "-o", str(tmp_path / "use.o")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


STEPS = (ctypes.c_float * 6)(3.4, -4.7, 2.0, 3.4, -4.7, 2.0)
BAD = (ctypes.c_float * 6)(3.4, -4.7, 2.0, 3.4, math.inf, 2.0)
ARGS = dict(batch=3, rows=8, cols=12, G=P, ldg=12, stride_g=96, O=P, ldo=12, stride_o=96, dtype=0, steps=2,
            coefficients=STEPS, eps=1e-7)


@pytest.mark.parametrize("change,code", [
    ({}, 0),
    ({"dtype": 2}, 0),
    ({"dtype": 1}, -1),
    ({"steps": 0}, -1),
    ({"steps": 33}, -1),
    ({"coefficients": None}, -1),
    ({"coefficients": BAD}, -1),
    ({"coefficients": BAD, "steps": 1}, 0),
    ({"eps": -1.0}, -1),
    ({"eps": math.nan}, -1),
    ({"eps": math.inf}, -1),
    ({"eps": 0.0}, 0),
    ({"batch": -1}, -1),
    ({"rows": -1}, -1),
    ({"cols": (1 << 20) + 1, "ldg": 1 << 21, "ldo": 1 << 21}, -1),
    ({"ldg": 11}, -1),
    ({"ldo": 11}, -1),
    ({"ldg": 1 << 37}, -1),
    ({"rows": 1 << 20, "ldg": 1 << 25, "stride_g": 1 << 45}, -1),
    ({"stride_g": 95}, -1),
    ({"stride_o": 95}, -1),
    ({"stride_o": 1 << 43}, -1),
    ({"batch": 1, "stride_g": 0, "stride_o": 0}, 0),
    ({"G": 0}, -1),
    ({"O": 0}, -1),
    ({"G": P + 2}, -2),
    ({"O": P + 2}, -2),
    ({"O": P + 2, "dtype": 2}, 0),
    ({"G": P + 1, "dtype": 2}, -2),
    ({"batch": 0, "G": 0, "O": 0}, 0),
    ({"rows": 0, "G": 0, "O": 0}, 0),
])
def test_arguments(g, change, code):
    assert g.gemm_orthogonalise_validate(*{**ARGS, **change}.values()) == code


def test_a_call_without_a_handle_is_refused(g):
    assert g.gemm_orthogonalise(None, *ARGS.values(), None) == g.GEMM_ERR_INVALID


def test_step_tables(g):
    assert list(g._step_table(2, (1, 2, 3))) == [1, 2, 3, 1, 2, 3]
    assert list(g._step_table(2, [(1, 2, 3), (4, 5, 6)])) == [1, 2, 3, 4, 5, 6]
    assert list(g._step_table(3, torch.arange(9.0).view(3, 3).tolist())) == list(range(9))
    for steps, c in ((0, (1, 2, 3)), (33, (1, 2, 3)), (2, [(1, 2, 3)]), (1, [(1, 2)]), (2, (1, 2))):
        with pytest.raises(ValueError):
            g._step_table(steps, c)


def test_cpu_tensors_are_refused(g):
    with pytest.raises(ValueError, match="CUDA device"):
        g.orthogonalise(torch.zeros(4, 4))
