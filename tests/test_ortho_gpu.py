"""Orthogonalised updates on the GPU against the steps in 64 bits.

Tolerances, of the result's norm.  A step has three products.  BF16: an operand's
FP16 rounding is at most 2^-11 of it, so 15 roundings of five steps stay within
15 * 2^-11 where the steps do not amplify them (what they do amplify, X itself, is
kept in two FP16 numbers), and the result's own rounding within 2^-8.  FP32: an
operand of two FP16 numbers is off by 2^-22, a sum's segments drop up to 2^-23 at
each of 48 additions, in sequence of random size 2^-24 * sqrt(48): 7e-7 a
product, sqrt(15) of that over five steps, amplified by the polynomial's slope
(at most a = 3.4445, once): 1e-5.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

USUAL = (3.4445, -4.7750, 2.0315)
TOL = {torch.bfloat16: 15 * 2.0 ** -11 + 2.0 ** -8, torch.float32: 1e-5}


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


def definition(G, steps=5, coefficients=USUAL, eps=1e-7):
    rows = [coefficients] * steps if not hasattr(coefficients[0], "__len__") else coefficients
    X = G.double().cpu()
    X = X / (X.square().sum((-2, -1), keepdim=True).sqrt() + eps)
    turned = X.shape[-2] > X.shape[-1]
    X = X.mT if turned else X
    for a, b, c in rows:
        A = X @ X.mT
        X = a * X + (b * A + c * A @ A) @ X
    return X.mT if turned else X


def updates(shape, dtype, seed, kind="few"):
    """Gradients: noise, or a few strong directions and noise."""
    gen = torch.Generator().manual_seed(seed)
    noise = torch.randn(shape, generator=gen)
    if kind == "noise":
        return noise.to(dtype)
    rank = max(1, min(shape[-2:]) // 8)
    left = torch.randn((*shape[:-1], rank), generator=gen) * torch.logspace(0, -2, rank)
    right = torch.randn((*shape[:-2], rank, shape[-1]), generator=gen)
    return ((left @ right / rank ** 0.5 + 0.03 * noise) * 1e-3).to(dtype)


def assert_near(out, want, dtype, times=1.0):
    assert out.dtype == dtype
    got = out.double().cpu()
    assert torch.isfinite(got).all()
    off = (got - want).norm(dim=(-2, -1))
    assert (off <= times * TOL[dtype] * want.norm(dim=(-2, -1))).all(), float((off / want.norm(dim=(-2, -1))).max())


SHAPES = [(1, 1), (1, 7), (7, 1), (2, 3), (31, 33), (63, 65), (64, 64), (65, 63), (127, 129), (130, 520), (520, 130),
          (256, 384), (300, 300), (513, 257)]


@pytest.mark.parametrize("kind", ["noise", "few"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}x{s[1]}")
def test_orthogonalise(gm, h, shape, dtype, kind):
    G = updates(shape, dtype, 1, kind)
    out = torch.full(shape, 7.0, dtype=dtype, device="cuda")
    h.orthogonalise(G.cuda(), out)
    h.sync_status()
    assert_near(out, definition(G), dtype)


@pytest.mark.parametrize("tile", [1032, 1064, 1128, 1256, 2032, 2064, 2128, 2256])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", [(3, 200, 330), (2, 600, 270)], ids=lambda s: f"{s[1]}x{s[2]}")
def test_every_tile(gm, h, shape, dtype, tile):
    """Several tiles a CTA, in batches."""
    h.set_option(gm.GEMM_OPT_ORTHO_TILE, tile)
    h.set_option(gm.GEMM_OPT_MAX_CTAS, 4)
    G = updates(shape, dtype, 2)
    out = torch.empty(shape, dtype=dtype, device="cuda")
    h.orthogonalise(G.cuda(), out)
    h.sync_status()
    assert_near(out, definition(G), dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_large_matrix(gm, h, dtype):
    G = updates((1000, 2100), dtype, 3)
    out = torch.empty_like(G, device="cuda")
    h.orthogonalise(G.cuda(), out)
    h.sync_status()
    assert_near(out, definition(G.cuda().double()), dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", [(40, 300, 400), (30, 500, 290)])
def test_many_matrices_of_different_norms(gm, h, shape, dtype):
    G = updates(shape, dtype, 23)
    G = (G.float() * (2.0 ** (torch.arange(shape[0]) % 9 - 4))[:, None, None]).to(dtype)
    out = torch.empty_like(G, device="cuda")
    h.orthogonalise(G.cuda(), out)
    h.sync_status()
    assert_near(out, definition(G.cuda().double()), dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_one_step_and_coefficients_of_each(gm, h, dtype):
    G = updates((70, 90), dtype, 4)
    out = torch.empty_like(G, device="cuda")
    for steps, c in ((1, USUAL), (1, (1.5, -0.5, 0.0)), (1, (0.0, 1.0, 0.0)), (2, USUAL), (8, (1.875, -1.25, 0.375)),
                     (3, [(4.0, -6.0, 3.0), (3.9, -5.5, 2.4), (1.875, -1.25, 0.375)])):
        h.orthogonalise(G.cuda(), out, steps, c)
        h.sync_status()
        assert_near(out, definition(G, steps, c), dtype, 2.0 if steps > 5 else 1.0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("turned", [False, True])
def test_strides_batches_and_in_place(gm, h, dtype, turned):
    rows, cols = (90, 70) if turned else (70, 90)
    G = updates((3, rows, cols), dtype, 5)
    want = definition(G)
    big = torch.full((3, 100, 101), 5.0, dtype=dtype, device="cuda")
    view = big[:, 3:3 + rows, 5:5 + cols]
    view.copy_(G)
    store = torch.full((3, 95, 97), 6.0, dtype=dtype, device="cuda")
    out = store[:, 1:1 + rows, 3:3 + cols]
    h.orthogonalise(view, out)
    h.sync_status()
    assert_near(out, want, dtype)
    rest = store.clone()
    rest[:, 1:1 + rows, 3:3 + cols] = 6
    assert (rest == 6).all()
    first = out.clone()
    h.orthogonalise(view, view)
    h.sync_status()
    assert torch.equal(view, first)  # bit for bit, in place and at another alignment
    rest = big.clone()
    rest[:, 3:3 + rows, 5:5 + cols] = 5
    assert (rest == 5).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_scales_of_every_magnitude(gm, h, dtype):
    """The result does not depend on G's scale, down to where eps counts (at
    2^-15 it is 7e-5 of the norm)."""
    G = updates((40, 64), dtype, 6, "noise").float()
    want = definition(G.to(dtype))
    for scale in (2.0 ** 120, 2.0 ** 60, 1.0, 2.0 ** -15):
        x = (G * scale).to(dtype)
        out = torch.empty((40, 64), dtype=dtype, device="cuda")
        h.orthogonalise(x.cuda(), out)
        h.sync_status()
        assert_near(out, definition(x), dtype)
    for scale, eps in ((2.0 ** -60, 0.0), (2.0 ** -120, 0.0)):
        h.orthogonalise((G * scale).to(dtype).cuda(), out, eps=eps)
        h.sync_status()
        assert_near(out, want, dtype)
    for scale in (2.0 ** -25, 2.0 ** -30, 2.0 ** -45, 2.0 ** -80):
        x = (G * scale).to(dtype)
        h.orthogonalise(x.cuda(), out)
        h.sync_status()
        assert_near(out, definition(x), dtype, 4.0)  # FP16's range is partly used up by the growth


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_odd_matrices_of_a_batch(gm, h, dtype, bad):
    """Zeros give zeros, what is not finite NaN, and neighbours are not touched."""
    G = updates((4, 150, 100), dtype, 7)
    G[1] = 0
    G[2, 149, 99] = bad
    out = torch.full(G.shape, 7.0, dtype=dtype, device="cuda")
    h.orthogonalise(G.cuda(), out)
    h.sync_status()
    assert (out[1] == 0).all() and torch.isnan(out[2]).all()
    assert_near(out[[0, 3]], definition(G[[0, 3]]), dtype)
    zeros = torch.zeros((3, 5), dtype=dtype, device="cuda")
    h.orthogonalise(zeros, zeros, eps=0.0)
    assert (zeros == 0).all()


def test_rows_of_different_sizes(gm, h):
    """Rows a million times smaller than others still come out as the steps say."""
    G = updates((64, 128), torch.float32, 8, "noise")
    G[::2] *= 1e-4
    out = torch.empty_like(G, device="cuda")
    h.orthogonalise(G.cuda(), out)
    h.sync_status()
    want = definition(G)
    assert_near(out, want, torch.float32)
    small = (out[::2].double().cpu() - want[::2]).norm() / want[::2].norm()
    assert small <= 1e-3


def test_a_batch_in_parts(gm, h):
    """A workspace limit that holds two of five matrices."""
    G = updates((5, 256, 320), torch.bfloat16, 9)
    whole, parts = (torch.empty(G.shape, dtype=G.dtype, device="cuda") for _ in range(2))
    h.orthogonalise(G.cuda(), whole)
    with gm.Gemm(0) as small:
        small.set_option(gm.GEMM_OPT_WORKSPACE_LIMIT, 2_600_000)
        small.orthogonalise(G.cuda(), parts)
        small.sync_status()
        assert torch.equal(parts, whole)
        small.set_option(gm.GEMM_OPT_WORKSPACE_LIMIT, 1)
    with gm.Gemm(0) as none:
        none.set_option(gm.GEMM_OPT_WORKSPACE_LIMIT, 1000)
        with pytest.raises(gm.GemmError) as e:
            none.orthogonalise(G.cuda(), parts)
        assert e.value.code == gm.GEMM_ERR_NOMEM


def test_streams_and_captured_graphs(gm, h):
    xs = [updates((2, 200, 160), torch.bfloat16, 10 + i).cuda() for i in range(3)]
    want = []
    for x in xs:
        out = torch.empty_like(x)
        h.orthogonalise(x, out)
        want.append(out)
    torch.cuda.synchronize()
    outs = [torch.empty_like(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(4):
        for x, o, s in zip(xs, outs, streams):
            h.orthogonalise(x, o, stream=s)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)
    with gm.Gemm(0) as fresh:  # its first call is captured
        static, out = xs[0].clone(), torch.empty_like(xs[0])
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            fresh.orthogonalise(static, out)
        for x, w in zip(xs, want):
            static.copy_(x)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, w)
        fresh.sync_status()


def test_expired_wait_is_reported_and_the_handle_recovers(gm, h):
    G = updates((2, 300, 400), torch.bfloat16, 13)
    want = definition(G)
    out = torch.empty(G.shape, dtype=G.dtype, device="cuda")
    h.set_option(gm.GEMM_OPT_WAIT_TIMEOUT_NS, 5_000_000)
    for tile in (1128, 2256):
        h.set_option(gm.GEMM_OPT_ORTHO_TILE, tile)
        h.set_option(gm.GEMM_OPT_DEBUG_DROP_LOAD, 1)
        h.orthogonalise(G.cuda(), out)
        with pytest.raises(gm.GemmError) as e:
            h.sync_status()
        assert e.value.code == gm.GEMM_ERR_TIMEOUT
        h.set_option(gm.GEMM_OPT_DEBUG_DROP_LOAD, 0)
        h.orthogonalise(G.cuda(), out)
        h.sync_status()
        assert_near(out, want, torch.bfloat16)


def test_module_function_and_refusals(gm, h):
    G = updates((50, 60), torch.bfloat16, 14).cuda()
    assert_near(gm.orthogonalise(G), definition(G), torch.bfloat16)
    assert gm.orthogonalise(G, out=G, handle=h) is G
    for call in (lambda: h.orthogonalise(G, G.float()), lambda: h.orthogonalise(G, G[:49]),
                 lambda: h.orthogonalise(G.half(), G.half()), lambda: h.orthogonalise(G, G, steps=0),
                 lambda: h.orthogonalise(G, G, coefficients=(1, 2)), lambda: h.orthogonalise(G.t(), G.t()),
                 lambda: h.orthogonalise(G, G[:1].expand(50, 60)), lambda: h.orthogonalise(G[None], G)):
        with pytest.raises(ValueError):
            call()
    for value in (3, 1000, 1224, 3064, 2512, -1):
        with pytest.raises(gm.GemmError):
            h.set_option(gm.GEMM_OPT_ORTHO_TILE, value)
    empty = torch.empty((0, 5), device="cuda")
    h.orthogonalise(empty, empty)
    assert h.last_path == "noop"


def test_update_of_expert_weights(gm):
    """The weight gradient of a grouped product, orthogonalised as a batch: near-
    orthogonal rows for every expert that had tokens, zeros for one that had none."""
    from dense_gemm_sm100_gb300.experts import grouped_matmul
    gen = torch.Generator().manual_seed(15)
    sizes, K, N = [300, 0, 200], 96, 64
    offsets = torch.tensor([0, 300, 300, 500], device="cuda")
    x = torch.randn((sum(sizes), K), generator=gen).bfloat16().cuda()
    w = torch.randn((3, K, N), generator=gen).bfloat16().cuda().requires_grad_()
    y = grouped_matmul(x, w, offsets)
    y.backward(torch.randn(y.shape, generator=gen).bfloat16().cuda())
    o = gm.orthogonalise(w.grad)
    assert (o[1] == 0).all()
    assert_near(o[[0, 2]], definition(w.grad[[0, 2]]), torch.bfloat16)
    values = torch.linalg.svdvals(o[[0, 2]].float())
    assert values.max() < 1.3 and values.median() > 0.6
