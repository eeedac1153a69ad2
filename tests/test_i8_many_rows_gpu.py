"""Quantisation to 8 bits where a CTA takes one row after another: codes and
scales bit for bit against the definition in FP64 (computed on the GPU by torch).

The grid holds at most 2048 threads an SM, so that rows follow one another in a
CTA from about 9700 rows on for up to 1024 columns, 1200 for up to 4096 and 300
above 8192.  Row counts leave the last round part-filled, column counts leave the
last 16 bytes part-filled.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dense_gemm_sm100_gb300 import build, gemm
    build.build()
    return gemm


@pytest.fixture()
def h(gm):
    with gm.Gemm(0) as handle:
        yield handle


def sample(rows, K, dtype, seed):
    """Normal values, each row at a scale of its own, a row of zeros among them and
    one that is not finite."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((rows, K), generator=gen, device="cuda")
    x *= torch.exp2(torch.randint(-20, 20, (rows, 1), generator=gen, device="cuda").float())
    x[rows // 2] = 0
    x[rows - 2, K - 1] = float("inf")
    return x.to(dtype)


def check(q, x):
    """Row blocks, so that the 64-bit copies stay small."""
    K = x.shape[1]
    for r in range(0, x.shape[0], 4096):
        v = x[r:r + 4096].double()
        fine = torch.isfinite(v).all(1)
        top = torch.where(fine, torch.nan_to_num(v).abs().amax(1), float("nan"))
        scales = (top / 127).float()
        got = q.scales[r:r + 4096]
        assert torch.equal(torch.isnan(got), ~fine) and torch.equal(got[fine], scales[fine])
        codes = torch.round(v / scales.double()[:, None]).clamp(-127, 127)
        codes = torch.where((scales > 0)[:, None], codes, torch.zeros_like(codes))
        assert torch.equal(q.codes[r:r + 4096, :K].double(), codes)
    assert (q.codes[:, K:] == 99).all()


SHAPES = [(30001, 250), (30001, 1000), (20003, 1021), (5003, 2040), (5003, 4088), (4001, 3001), (2503, 8184),
          (2047, 5003), (1501, 16376), (1203, 9001), (803, 20007)]


def storage(gm, rows, K):
    q = gm.i8_empty(rows, K)
    q.codes.fill_(99)
    q.scales.fill_(-9)
    return q


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}x{s[1]}")
def test_rows_on_16_byte_boundaries(gm, h, shape, dtype):
    rows, K = shape
    pitch = (K + 15) // 16 * 16
    x = torch.full((rows, pitch), float("nan"), dtype=dtype, device="cuda")  # what is behind a row does not count
    x[:, :K] = sample(rows, K, dtype, 1)
    q = storage(gm, rows, K)
    h.i8_quantise(x[:, :K], q)
    h.sync_status()
    check(q, x[:, :K])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}x{s[1]}")
def test_rows_anywhere(gm, h, shape, dtype):
    rows, K = shape
    x = torch.full((rows, K + 3), float("nan"), dtype=dtype, device="cuda")
    x[:, 1:K + 1] = sample(rows, K, dtype, 2)
    q = storage(gm, rows, K)
    h.i8_quantise(x[:, 1:K + 1], q)
    h.sync_status()
    check(q, x[:, 1:K + 1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("batch,rows,K", [(31, 999, 248), (7, 701, 4088), (5, 301, 16376)])
def test_batches(gm, h, batch, rows, K, dtype):
    """Rows of one CTA that belong to different matrices of a batch."""
    x = torch.full((batch, rows + 5, K + 8), float("nan"), dtype=dtype, device="cuda")
    view = x[:, :rows, :K]
    view.copy_(sample(batch * rows, K, dtype, 3).view(batch, rows, K))
    q = storage(gm, batch * rows, K)
    h.i8_quantise(view, q)
    h.sync_status()
    check(q, view.reshape(batch * rows, K))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", [(30001, 250), (5003, 2040), (9001, 777)], ids=lambda s: f"{s[0]}x{s[1]}")
def test_row_major_and_back(gm, h, shape, dtype):
    """Column-wise quantisation and the inverse, over many CTAs."""
    rows, K = shape
    x = sample(rows, K, dtype, 4)
    q = storage(gm, rows, K)
    h.i8_quantise(x.t().contiguous(), q, "row")
    h.sync_status()
    check(q, x)
    out = torch.empty((rows, K), dtype=dtype, device="cuda")
    h.i8_dequantise(q, out)
    want = (q.codes[:, :K].float() * q.scales[:, None]).to(dtype)
    assert torch.equal(torch.isnan(out), torch.isnan(want)) and torch.equal(torch.nan_to_num(out), torch.nan_to_num(want))
