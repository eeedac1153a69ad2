"""The grouped and 4-bit entry points without a GPU: declared functions are
exported, the headers are plain C, arguments are checked on the host."""
import os
import re
import shutil
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADERS = [os.path.join(ROOT, "include", n) for n in ("gemm_grouped.h", "gemm_mx4.h")]
P = 0x10000  # a fake, aligned address: the checks never dereference


@pytest.fixture(scope="module")
def g():
    from dense_gemm_sm100_gb300 import build, gemm
    build.build()
    gemm.load_library()
    return gemm


def test_declared_functions_are_exported_and_bound(g):
    lib = g.load_library()
    names = set()
    for h in HEADERS:
        names.update(re.findall(r"\b(gemm_[a-z0-9_]+)\s*\(", re.sub(r"/\*.*?\*/", "", open(h).read(), flags=re.S)))
    assert len(names) == 13
    for n in names:
        assert hasattr(lib, n) and hasattr(g, n), n


def test_headers_are_plain_c(tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("no gcc")
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    src = tmp_path / "use.c"
    src.write_text('#include "gemm_grouped.h"\n#include "gemm_mx4.h"\n'
                   "int main(void) { return GEMM_MX4_BLOCK == 32 && GEMM_GROUPED_MAX_GROUPS > 0 ? 0 : 1; }\n")
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"),
                        "-isystem", os.path.join(cuda, "include"), "-c", str(src), "-o", str(tmp_path / "use.o")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


# layout, groups, rows, N, K, offsets, A, lda, B, ldb, stride_b, C, ldc, dtype, c_dtype
GROUPED = dict(layout=0, groups=3, rows=8, N=4, K=6, offsets=P, A=P, lda=6, B=P, ldb=4, stride_b=24, C=P, ldc=4,
               dtype=2, c_dtype=0)


@pytest.mark.parametrize("change,code", [
    ({}, 0),
    ({"layout": 1, "ldb": 6}, 0),
    ({"c_dtype": 2}, 0),
    ({"dtype": 1}, 0),
    ({"layout": 2}, -1),
    ({"dtype": 0}, -1),                      # FP32 SIMT has no grouped form
    ({"dtype": 3}, -1),
    ({"dtype": 1, "c_dtype": 2}, -1),        # TF32 writes float
    ({"c_dtype": 1}, -1),
    ({"groups": 0}, -1),
    ({"groups": 4097}, -1),
    ({"rows": -1}, -1),
    ({"K": -1}, -1),
    ({"offsets": 0}, -1),
    ({"offsets": P + 4}, -2),
    ({"A": 0}, -1),
    ({"C": 0}, -1),
    ({"lda": 5}, -1),
    ({"ldb": 3}, -1),
    ({"ldc": 3}, -1),
    ({"stride_b": 23}, -1),                  # groups overlap
    ({"groups": 1, "stride_b": 0}, 0),       # one group has no stride
    ({"stride_b": 1 << 38}, -1),
    ({"A": P + 1}, -2),
    ({"A": P + 2}, 0),                       # re-packed
    ({"dtype": 1, "A": P + 2}, -2),
    ({"C": P + 2}, -2),
    ({"C": P + 2, "c_dtype": 2}, 0),
    ({"rows": 0, "A": 0, "C": 0}, 0),
    ({"N": 0, "B": 0, "C": 0}, 0),
    ({"K": 0, "A": 0, "B": 0}, 0),
    ({"rows": 1 << 31}, -1),
    ({"rows": 1 << 30, "lda": 1 << 36}, -1),             # rows times pitch past any memory
    ({"K": 1 << 30, "lda": 1 << 30, "ldb": 1 << 36, "stride_b": 1 << 37}, -1),
    ({"rows": 1 << 30, "ldc": 1 << 36}, -1),
    ({"rows": (1 << 31) - 2048, "N": (1 << 31) - 2048, "ldc": 1 << 31, "ldb": 1 << 31, "stride_b": 1 << 36}, -1),
])
def test_grouped_arguments(g, change, code):
    assert g.gemm_grouped_validate(*{**GROUPED, **change}.values()) == code


# groups, rows, M, N, offsets, A, lda, B, ldb, C, ldc, stride_c, dtype, c_dtype
WGRAD = dict(groups=3, rows=8, M=4, N=6, offsets=P, A=P, lda=4, B=P, ldb=6, C=P, ldc=6, stride_c=24, dtype=2, c_dtype=0)


@pytest.mark.parametrize("change,code", [
    ({}, 0),
    ({"dtype": 1}, 0),
    ({"dtype": 0}, -1),
    ({"groups": 0}, -1),
    ({"offsets": 0}, -1),
    ({"lda": 3}, -1),
    ({"ldb": 5}, -1),
    ({"ldc": 5}, -1),
    ({"stride_c": 23}, -1),
    ({"groups": 1, "stride_c": 0}, 0),
    ({"B": 0}, -1),
    ({"B": P + 1}, -2),
    ({"C": P + 1, "c_dtype": 2}, -2),
    ({"rows": 0, "A": 0, "B": 0}, 0),        # every C is zero
    ({"M": 0, "C": 0}, 0),
    ({"M": 1 << 30, "lda": 1 << 30, "ldc": 1 << 36, "stride_c": 1 << 37}, -1),
])
def test_wgrad_arguments(g, change, code):
    assert g.gemm_grouped_wgrad_validate(*{**WGRAD, **change}.values()) == code


# groups, rows, N, K, offsets, codes, pitch, scales, pitch (A, then B), C, ldc, c_dtype
MX4 = dict(groups=2, rows=4, N=5, K=40, offsets=P, ac=P, aq=32, as_=P, al=16, bc=P, bq=32, bs=P, bl=16, C=P, ldc=5,
           c_dtype=0)


@pytest.mark.parametrize("change,code", [
    ({}, 0),
    ({"groups": 1, "offsets": 0}, 0),        # the dense product
    ({"offsets": 0}, -1),
    ({"c_dtype": 1}, -1),
    ({"aq": 16}, -1),                        # 40 elements pad to 64: 32 bytes
    ({"aq": 40}, -2),
    ({"al": 0}, -1),
    ({"bl": 8}, -2),
    ({"bc": P + 8}, -2),
    ({"as_": 0}, -1),
    ({"C": P + 2}, -2),
    ({"ldc": 4}, -1),
    ({"K": 0, "ac": 0, "bc": 0}, 0),
    ({"rows": 0, "C": 0}, 0),
    ({"groups": 4096, "N": 1 << 20, "ldc": 1 << 20}, -1),
    ({"N": 1 << 20, "ldc": 1 << 20, "bq": 1 << 30}, -1),
])
def test_mx4_arguments(g, change, code):
    assert g.gemm_mx4_validate(*{**MX4, **change}.values()) == code


# layout, batch, rows, K, src, ld, stride, src_dtype, codes, ldq, scales, lds
QUANT = dict(layout=1, batch=1, rows=4, K=40, src=P, ld=40, stride=0, dtype=2, codes=P, ldq=32, scales=P, lds=16)


@pytest.mark.parametrize("change,code", [
    ({}, 0),
    ({"layout": 0, "ld": 4}, 0),
    ({"layout": 0, "ld": 3}, -1),
    ({"ld": 39}, -1),
    ({"dtype": 1}, -1),
    ({"batch": 2, "stride": 160}, 0),
    ({"batch": 2, "stride": 159}, -1),
    ({"src": P + 1}, -2),
    ({"ldq": 16}, -1),
    ({"scales": P + 1}, -2),
    ({"rows": 0, "src": 0}, 0),
    ({"rows": 1 << 30, "ld": 1 << 36}, -1),
])
def test_quantise_arguments(g, change, code):
    assert g.gemm_mx4_quantise_validate(*{**QUANT, **change}.values()) == code


def test_dequantise_arguments(g):
    ok = [4, 40, P, 32, P, 16, P, 40, 0]
    assert g.gemm_mx4_dequantise_validate(*ok) == 0
    assert g.gemm_mx4_dequantise_validate(*ok[:7], 39, 0) == -1
    assert g.gemm_mx4_dequantise_validate(*ok[:6], P + 2, 40, 0) == -2
    assert g.gemm_mx4_dequantise_validate(*ok[:8], 1) == -1


def test_pitches(g):
    assert [g.gemm_mx4_code_pitch(k) for k in (0, 1, 32, 33, 1000, 4096)] == [0, 16, 16, 32, 512, 2048]
    assert [g.gemm_mx4_scale_pitch(k) for k in (0, 1, 512, 513, 4096)] == [0, 16, 16, 32, 128]


def test_null_handle_is_refused(g):
    assert g.gemm_grouped_run(None, *GROUPED.values(), None) == g.GEMM_ERR_INVALID
    assert g.gemm_grouped_wgrad(None, *WGRAD.values(), None) == g.GEMM_ERR_INVALID
    assert g.gemm_mx4_grouped_run(None, *MX4.values(), None) == g.GEMM_ERR_INVALID
    assert g.gemm_mx4_quantise(None, *QUANT.values(), None) == g.GEMM_ERR_INVALID


def test_mx4_storage_is_checked(g):
    q = g.mx4_empty(3, 1000, device="cpu")
    assert q.codes.shape == (3, 512) and q.scales.shape == (3, 32) and (q.rows, q.K) == (3, 1000)
    with pytest.raises(ValueError):
        g.Mx4(q.codes, q.scales, 2000)
    with pytest.raises(ValueError):
        g.Mx4(q.codes.to(torch.int32), q.scales, 1000)
    with pytest.raises(ValueError):
        g.Mx4(q.codes, q.scales[:2], 1000)


def test_group_rows_sorts_and_counts():
    from dense_gemm_sm100_gb300.experts import group_rows
    expert = torch.tensor([3, 1, 1, 0, 3, 5, 1])
    order, offsets = group_rows(expert, 7)
    assert order.tolist() == [3, 1, 2, 6, 0, 4, 5]
    assert offsets.tolist() == [0, 1, 4, 4, 6, 6, 7, 7] and offsets.dtype == torch.int64
    order, offsets = group_rows(expert[:0], 2)
    assert order.numel() == 0 and offsets.tolist() == [0, 0, 0]


def test_grouped_matmul_needs_a_gpu_tensor():
    from dense_gemm_sm100_gb300.experts import grouped_matmul
    with pytest.raises(ValueError):
        grouped_matmul(torch.zeros(2, 3), torch.zeros(1, 3, 4), torch.tensor([0, 2]))


def test_mx4_rows_closer_together_than_their_columns(g):
    """Rows of 32 bytes of codes 32 bytes apart, seen as 64 columns: the pitch is
    the distance of the rows, or reads run past the end of the storage."""
    codes = torch.zeros(4 * 32 + 32, dtype=torch.uint8).as_strided((4, 64), (32, 1))
    scales = torch.zeros(4 * 16 + 16, dtype=torch.uint8).as_strided((4, 32), (16, 1))
    q = g.Mx4(codes, scales, 64)
    q._device = 0
    assert q._args(0)[1::2] == (32, 16)
    one = g.Mx4(codes[:1], scales[:1], 64)  # one row has no distance: the columns that it shows
    one._device = 0
    assert one._args(0)[1::2] == (64, 32)
    wide = g.Mx4(torch.zeros(4, 64, dtype=torch.uint8)[:, :32], torch.zeros(4, 48, dtype=torch.uint8)[:, :16], 64)
    wide._device = 0
    assert wide._args(0)[1::2] == (64, 48)


def test_the_nan_flag_is_taken_with_a_weight_gradients_type(g):
    for c_dtype in (g.GEMM_F32, g.GEMM_BF16):
        flagged = {"c_dtype": c_dtype | g.GEMM_GROUPED_NAN_ON_ERROR}
        assert g.gemm_grouped_wgrad_validate(*{**WGRAD, **flagged}.values()) == 0
        assert g.gemm_grouped_validate(*{**GROUPED, **flagged}.values()) == -1
        assert g.gemm_mx4_validate(*{**MX4, **flagged}.values()) == -1
    assert g.gemm_grouped_wgrad_validate(*{**WGRAD, "c_dtype": 1 | g.GEMM_GROUPED_NAN_ON_ERROR}.values()) == -1
    assert g.gemm_grouped_wgrad_validate(*{**WGRAD, "dtype": 1, "c_dtype": 2 | g.GEMM_GROUPED_NAN_ON_ERROR}.values()) == -1
