"""Orthogonalised updates of matrices far below eps, over many steps, against the
steps in 64 bits.

Such a matrix grows by a step's a until its products hold it back.  Tolerances
follow the singular values of the exact steps.  A step s -> f(s) = a s + b s^3 + c s^5
passes an error on with at most L = max(|f'|, f / s) over the singular values, and adds,
with operands that are off by u of themselves, at most u (5 |b| S^2 + 8 |c| S^4) of X's
norm (S the largest singular value; A takes X twice and is rounded, A A takes A twice,
B is rounded, and X once more), and 2^-20 for what X itself loses (two FP16 numbers)
and the factors.  u is FP16's half step 2^-11 for BF16 results; for FP32 results two
FP16 numbers, and sums of at most 260 products, are off by less than 7e-7.  The result
is rounded once, by at most 2^-8 or 2^-24 of itself.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

USUAL = (3.4445, -4.7750, 2.0315)
SLOW = (1.875, -1.25, 0.375)  # f'(1) = 0: errors are not passed on
UNIT = {torch.bfloat16: 2.0 ** -11, torch.float32: 7e-7}
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


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


def definition(G, rows, eps):
    """(X, bound on the error of a computed X relative to its norm)."""
    X = G.double()
    X = X / (X.norm() + eps)
    turned = X.shape[0] > X.shape[1]
    X = X.mT if turned else X
    bounds = {t: 0.0 for t in UNIT}
    for a, b, c in rows:
        s = torch.linalg.svdvals(X)
        s = s[s > 1e-9 * s[0]] if s[0] > 0 else s[:1]
        grid = torch.cat([s, torch.linspace(float(s.min()), float(s.max()), 200, dtype=torch.float64)])
        slope = (a + 3 * b * grid ** 2 + 5 * c * grid ** 4).abs()
        passed = float(torch.maximum(slope, (a + b * grid ** 2 + c * grid ** 4).abs()).max())
        S = float(s.max())
        A = X @ X.mT
        new = a * X + (b * A + c * A @ A) @ X
        ratio = float(X.norm() / new.norm())
        for t, u in UNIT.items():
            bounds[t] = ratio * (passed * bounds[t] + u * (5 * abs(b) * S ** 2 + 8 * abs(c) * S ** 4)) + 2.0 ** -20
        X = new
    return (X.mT if turned else X), {t: v + ROUND[t] for t, v in bounds.items()}


def check(out, G, rows, eps=1e-7):
    want, bounds = definition(G.cpu(), rows, eps)
    got = out.double().cpu()
    assert torch.isfinite(got).all()
    off = float((got - want).norm() / want.norm())
    assert off <= min(bounds[out.dtype], 0.5), (off, bounds[out.dtype])


def orthonormal(rows, cols, seed):
    """All singular values equal."""
    gen = torch.Generator().manual_seed(seed)
    q, _ = torch.linalg.qr(torch.randn((max(rows, cols), min(rows, cols)), generator=gen, dtype=torch.float64))
    return (q if rows >= cols else q.mT).contiguous()


NORMS = [1e-9, 1e-12, 1e-20, 1e-30]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("coefficients", [USUAL, SLOW], ids=["usual", "slow"])
@pytest.mark.parametrize("steps", [5, 8, 9, 10, 16, 32])
def test_one_entry(gm, h, steps, coefficients, dtype):
    """One entry that is not zero: its square is the diagonal of A, everything else is exact."""
    for shape, at in (((1, 1), (0, 0)), ((32, 32), (5, 7)), ((70, 40), (69, 3)), ((40, 300), (0, 299))):
        for norm in NORMS:
            G = torch.zeros(shape, dtype=dtype)
            G[at] = -norm
            out = torch.full(shape, 7.0, dtype=dtype, device="cuda")
            h.orthogonalise(G.cuda(), out, steps, coefficients)
            h.sync_status()
            check(out, G, [coefficients] * steps)
            rest = out.clone()
            rest[at] = 0
            assert (rest == 0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("steps", [5, 8, 10, 16, 32])
@pytest.mark.parametrize("shape", [(32, 48), (48, 32), (130, 260), (257, 120)], ids=lambda s: f"{s[0]}x{s[1]}")
def test_equal_singular_values(gm, h, shape, steps, dtype):
    for norm in NORMS:
        G = (orthonormal(*shape, 1) * (norm / min(shape) ** 0.5)).to(dtype)
        out = torch.full(shape, 7.0, dtype=dtype, device="cuda")
        h.orthogonalise(G.cuda(), out, steps, SLOW)
        h.sync_status()
        check(out, G, [SLOW] * steps)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("steps", [5, 8, 10, 12, 16])
def test_noise(gm, h, steps, dtype):
    gen = torch.Generator().manual_seed(2)
    for shape in ((32, 48), (100, 64)):
        noise = torch.randn(shape, generator=gen, dtype=torch.float64)
        for norm in (1e-9, 1e-11, 1e-14, 1e-20):
            G = (noise * (norm / noise.norm())).to(dtype)
            out = torch.full(shape, 7.0, dtype=dtype, device="cuda")
            h.orthogonalise(G.cuda(), out, steps)
            h.sync_status()
            check(out, G, [USUAL] * steps)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_large_first_coefficients(gm, h, dtype):
    """A schedule that grows by 8 a step, and one whose steps shrink in between."""
    for rows, norms in (([(8.0, -22.0, 16.0)] * 5 + [SLOW] * 3, (1e-10, 1e-12, 1e-15)),
                        ([(100.0, -50.0, 10.0)] * 3 + [SLOW] * 4, (5e-13, 1e-13, 1e-15)),
                        ([USUAL, (0.25, 0.0, 0.0)] * 4 + [USUAL] * 4, (1e-10, 1e-12, 1e-15))):
        for norm in norms:
            G = (orthonormal(40, 56, 3) * (norm / 40 ** 0.5)).to(dtype)
            out = torch.full((40, 56), 7.0, dtype=dtype, device="cuda")
            h.orthogonalise(G.cuda(), out, len(rows), rows)
            h.sync_status()
            check(out, G, rows)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tile", [0, 1032, 1128, 2064, 2256])
def test_a_batch_of_different_norms(gm, h, dtype, tile):
    """Every matrix of a batch as if it stood alone, the ones above eps too."""
    h.set_option(gm.GEMM_OPT_ORTHO_TILE, tile)
    norms = [1.0, 1e-9, 0.0, 1e-16, 1e3, 1e-12, 1e-30]
    base = orthonormal(70, 150, 4) / 70 ** 0.5
    G = torch.stack([base * n for n in norms]).to(dtype)
    for steps in (6, 12, 20):
        out = torch.full(G.shape, 7.0, dtype=dtype, device="cuda")
        h.orthogonalise(G.cuda(), out, steps, SLOW)
        again = torch.empty_like(out)
        h.orthogonalise(G.cuda(), again, steps, SLOW)
        h.sync_status()
        assert torch.equal(out, again)
        for i, n in enumerate(norms):
            if n == 0.0:
                assert (out[i] == 0).all()
                continue
            check(out[i], G[i], [SLOW] * steps)
            alone = torch.empty_like(out[i])
            h.orthogonalise(G[i].cuda(), alone, steps, SLOW)
            assert (alone.float() - out[i].float()).norm() <= 2 * (UNIT[dtype] * 40 + ROUND[dtype]) * out[i].float().norm()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_captured_with_other_norms(gm, h, dtype):
    """The powers of two belong to the data, not to the call: a replayed graph takes
    matrices of any norm."""
    base = orthonormal(64, 100, 5) / 8
    G = (base * 1e-3).to(dtype).cuda()
    out = torch.empty_like(G)
    h.orthogonalise(G, out, 12, SLOW)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h.orthogonalise(G, out, 12, SLOW)
    for norm in (1e-9, 1.0, 1e-13, 1e-25, 1e-2):
        G.copy_((base * norm).to(dtype))
        graph.replay()
        torch.cuda.synchronize()
        check(out, G, [SLOW] * 12)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_singular_values_of_almost_8(gm, h, dtype):
    """The largest that the stated range allows: an element off A's diagonal is half of
    the largest singular value's square."""
    G = torch.ones((2, 2), dtype=dtype)
    rows = [(7.9, 0.0, 0.0), (1.0, -0.01, 0.0)]
    out = torch.empty((2, 2), dtype=dtype, device="cuda")
    h.orthogonalise(G.cuda(), out, 2, rows)
    h.sync_status()
    check(out, G, rows)
