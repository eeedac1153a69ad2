"""The 8-bit entry points without a GPU: declared functions are exported, the
header is plain C, arguments are checked on the host."""
import os
import re
import shutil
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gemm_i8.h")
P = 0x10000  # a fake, aligned address: the checks never dereference


@pytest.fixture(scope="module")
def g():
    from dense_gemm_sm100_gb300 import build, gemm
    build.build()
    gemm.load_library()
    return gemm


def test_declared_functions_are_exported_and_bound(g):
    names = set(re.findall(r"\b(gemm_[a-z0-9_]+)\s*\(", re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)))
    assert len(names) == 8
    for n in names:
        assert hasattr(g.load_library(), n) and hasattr(g, n), n


def test_header_is_plain_c(tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("no gcc")
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    src = tmp_path / "use.c"
    src.write_text('#include "gemm_i8.h"\nint main(void) { return gemm_i8_code_pitch(17) == 32 ? 0 : 1; }\n')
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"),
                        "-isystem", os.path.join(cuda, "include"), "-c", str(src), "-o", str(tmp_path / "use.o")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_pitches(g):
    assert [g.gemm_i8_code_pitch(k) for k in (-1, 0, 1, 16, 17, 4096)] == [0, 0, 16, 16, 32, 4096]


QUANTISE = dict(layout=1, batch=3, rows=8, K=20, src=P, ld=20, stride=160, src_dtype=0, codes=P, ldq=32, scales=P)


@pytest.mark.parametrize("change,code", [
    ({}, 0),
    ({"layout": 0, "ld": 8}, 0),
    ({"src_dtype": 2}, 0),
    ({"src_dtype": 1}, -1),
    ({"layout": 2}, -1),
    ({"layout": 0, "ld": 7}, -1),
    ({"ld": 19}, -1),
    ({"stride": 159}, -1),
    ({"batch": 1, "stride": 0}, 0),
    ({"batch": -1}, -1),
    ({"batch": 1 << 20, "rows": 1 << 20, "stride": 1 << 30}, -1),
    ({"src": 0}, -1),
    ({"codes": 0}, -1),
    ({"scales": 0}, -1),
    ({"ldq": 16}, -1),
    ({"ldq": 24}, -2),
    ({"codes": P + 8}, -2),
    ({"scales": P + 2}, -2),
    ({"scales": P + 4}, 0),
    ({"src": P + 2}, -2),
    ({"src": P + 2, "src_dtype": 2}, 0),
    ({"K": 0, "src": 0, "codes": 0, "scales": 0}, 0),
    ({"rows": 1 << 30, "batch": 1, "ldq": 1 << 16}, -1),
])
def test_quantise_arguments(g, change, code):
    assert g.gemm_i8_quantise_validate(*{**QUANTISE, **change}.values()) == code


DEQUANTISE = dict(rows=8, K=20, codes=P, ldq=32, scales=P, dst=P, ldd=20, dst_dtype=0)


@pytest.mark.parametrize("change,code", [
    ({}, 0),
    ({"dst_dtype": 2, "dst": P + 2}, 0),
    ({"dst_dtype": 3}, -1),
    ({"dst": P + 2}, -2),
    ({"dst": 0}, -1),
    ({"ldd": 19}, -1),
    ({"ldq": 16}, -1),
    ({"ldq": 40}, -2),
    ({"rows": 0, "codes": 0, "scales": 0, "dst": 0}, 0),
    ({"rows": -1}, -1),
])
def test_dequantise_arguments(g, change, code):
    assert g.gemm_i8_dequantise_validate(*{**DEQUANTISE, **change}.values()) == code


PRODUCT = dict(groups=3, rows=8, N=5, K=20, offsets=P, ac=P, aq=32, asc=P, bc=P, bq=32, bsc=P, C=P, ldc=5, c_dtype=0)


@pytest.mark.parametrize("change,code", [
    ({}, 0),
    ({"groups": 1, "offsets": 0}, 0),        # the dense call
    ({"offsets": 0}, -1),
    ({"c_dtype": 2}, 0),
    ({"c_dtype": 1}, -1),
    ({"groups": 4097}, -1),
    ({"rows": -1}, -1),
    ({"rows": 1 << 31}, -1),
    ({"N": -1}, -1),
    ({"ac": 0}, -1),
    ({"asc": 0}, -1),
    ({"bc": 0}, -1),
    ({"bsc": 0}, -1),
    ({"aq": 16}, -1),
    ({"bq": 16}, -1),
    ({"aq": 40}, -2),
    ({"bc": P + 8}, -2),
    ({"bsc": P + 1}, -2),
    ({"asc": P + 4}, 0),
    ({"C": P + 2}, -2),
    ({"C": P + 2, "c_dtype": 2}, 0),
    ({"ldc": 4}, -1),
    ({"rows": 0, "ac": 0, "C": 0}, 0),
    ({"K": 0, "ac": 0, "bc": 0, "asc": 0, "bsc": 0}, 0),
    ({"groups": 4096, "N": 1 << 20, "ldc": 1 << 20}, -1),
    ({"groups": 2, "N": 1 << 25, "ldc": 1 << 25, "bq": 1 << 17}, -1),
])
def test_product_arguments(g, change, code):
    assert g.gemm_i8_validate(*{**PRODUCT, **change}.values()) == code


def test_calls_without_a_handle_are_refused(g):
    assert g.gemm_i8_quantise(None, *QUANTISE.values(), None) == g.GEMM_ERR_INVALID
    assert g.gemm_i8_dequantise(None, *DEQUANTISE.values(), None) == g.GEMM_ERR_INVALID
    assert g.gemm_i8_grouped_run(None, *PRODUCT.values(), None) == g.GEMM_ERR_INVALID
    dense = [PRODUCT[k] for k in ("rows", "N", "K", "ac", "aq", "asc", "bc", "bq", "bsc", "C", "ldc", "c_dtype")]
    assert g.gemm_i8_run(None, *dense, None) == g.GEMM_ERR_INVALID


def test_operand_checks(g):
    q = g.i8_empty(4, 20, device="cpu")
    assert q.codes.shape == (4, 32) and q.rows == 4 and q.K == 20
    with pytest.raises(ValueError, match="cpu"):
        q._args(0)
    for codes, scales, K in ((q.codes.to(torch.uint8), q.scales, 20), (q.codes[:, ::2], q.scales, 16),
                             (q.codes, q.scales, 33), (q.codes, q.scales[:3], 20), (q.codes, q.scales.double(), 20),
                             (q.codes[:1].expand(4, 32), q.scales, 20), (q.codes, torch.zeros(8)[::2], 20)):
        with pytest.raises(ValueError):
            g.I8(codes, scales, K)
