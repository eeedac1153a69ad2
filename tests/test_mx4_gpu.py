"""Microscaled 4-bit floating point on the GPU: quantisation bit for bit against
its definition in FP64, products element by element.

A product of two E2M1 values and their power-of-two scales is exact in FP32,
so |C - ref| <= (K + 2) 2^-23 S, S = sum |a b|; a BF16 result is the FP32 result
of the same call rounded once, bit for bit.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

GRID = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)


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


def definition(x):
    """(codes as integers, scale bytes, values) of a 2-D tensor, element by
    element from the definition: nearest grid value, ties to the even index."""
    rows, K = x.shape
    Kp = -(-K // 32) * 32
    x = torch.nn.functional.pad(x.double(), (0, Kp - K)).view(rows, -1, 32)
    codes = torch.zeros(x.shape, dtype=torch.int64)
    scales = torch.zeros(x.shape[:2], dtype=torch.int64)
    values = torch.full(x.shape, float("nan"), dtype=torch.float64)
    for r in range(rows):
        for b in range(x.shape[1]):
            v = x[r, b]
            if not torch.isfinite(v).all():
                scales[r, b] = 255
                continue
            top = float(v.abs().max())
            e = max(math.frexp(top)[1] - 3, -127) if top > 0 else -127
            scales[r, b] = e + 127
            a = v.abs() / 2.0 ** e
            d = (a[:, None] - GRID).abs()
            best = d.min(1, keepdim=True).values
            tie = d == best  # one or two neighbours: the even index wins
            idx = torch.where(tie.sum(1) > 1,
                              (tie * torch.tensor([1, 0, 1, 0, 1, 0, 1, 0])).argmax(1), tie.double().argmax(1))
            codes[r, b] = idx + 8 * torch.signbit(v)
            values[r, b] = torch.copysign(GRID[idx], v) * 2.0 ** e
    return codes.view(rows, Kp), scales, values.view(rows, Kp)[:, :K]


def unpack(q):
    Kp = -(-q.K // 32) * 32
    c = q.codes[:, :Kp // 2].cpu().long()
    return torch.stack((c % 16, c // 16), -1).view(q.rows, Kp), q.scales[:, :Kp // 32].cpu().long()


def quantise(gm, h, x, layout="col"):
    rows, K = x.shape
    q = gm.mx4_empty(rows, K)
    q.codes.fill_(0xAA)
    q.scales.fill_(0xAA)
    h.mx4_quantise((x if layout == "col" else x.t().contiguous()).cuda(), q, layout)
    return q


def sample(rows, K, dtype, seed, spread=4.0):
    """Normal values, each row and each block at a scale of its own."""
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, K), generator=gen)
    x = x * torch.exp2(torch.randint(-int(spread), int(spread) + 1, (rows, 1), generator=gen).float())
    blocks = torch.exp2(torch.randint(-3, 4, (rows, -(-K // 32)), generator=gen).float())
    return (x * blocks.repeat_interleave(32, 1)[:, :K]).to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["row", "col"])
@pytest.mark.parametrize("shape", [(1, 1), (3, 31), (2, 33), (40, 100), (5, 256), (9, 1000), (70, 520)])
def test_quantise_matches_the_definition(gm, h, shape, layout, dtype):
    x = sample(*shape, dtype, 1)
    q = quantise(gm, h, x, layout)
    codes, scales, values = definition(x)
    got_codes, got_scales = unpack(q)
    assert torch.equal(got_codes, codes) and torch.equal(got_scales, scales)
    out = torch.empty(shape, dtype=dtype, device="cuda")
    h.mx4_dequantise(q, out)
    h.sync_status()
    assert torch.equal(out.cpu().double(), values)
    Kp = -(-shape[1] // 32) * 32
    assert (q.codes[:, Kp // 2:] == 0xAA).all() and (q.scales[:, Kp // 32:] == 0xAA).all()


def test_ties_saturation_and_signs(gm, h):
    x = torch.zeros(6, 32)
    x[0, :8] = torch.tensor([4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])   # every tie, scale 1
    x[1, :8] = -x[0, :8]
    x[2, :5] = torch.tensor([7.9, 6.5, 6.0, 5.01, 4.99])                      # past 6: saturates
    x[3, :4] = torch.tensor([0.2500001, 0.2499999, 4.0, -0.0])
    x[4, :3] = torch.tensor([float.fromhex("0x1p-149"), 2.0 ** -140, -(2.0 ** -130)])  # subnormal
    x[5, :3] = torch.tensor([3.4e38, -1e38, 2.0 ** 100])
    for layout in ("col", "row"):
        q = quantise(gm, h, x, layout)
        codes, scales, _ = definition(x)
        got = unpack(q)
        assert torch.equal(got[0], codes) and torch.equal(got[1], scales)
    assert got[0][0, :8].tolist() == [6, 0, 2, 2, 4, 4, 6, 6] and got[0][2, :5].tolist() == [7, 7, 7, 7, 6]


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_block_that_is_not_finite_becomes_nan(gm, h, bad):
    x = sample(4, 96, torch.float32, 2)
    x[1, 40] = bad
    for layout in ("col", "row"):
        q = quantise(gm, h, x, layout)
        codes, scales = unpack(q)
        assert scales[1, 1] == 255 and (codes[1, 32:64] == 0).all() and (scales == 255).sum() == 1
        out = torch.empty((4, 96), device="cuda")
        h.mx4_dequantise(q, out)
        assert torch.isnan(out[1, 32:64]).all() and torch.isfinite(out).sum() == 4 * 96 - 32
        B = quantise(gm, h, sample(130, 96, torch.float32, 3))
        C = torch.empty((4, 130), device="cuda")
        h.run_mx4(q, B, C)
        h.sync_status()
        assert torch.isnan(C[1]).all() and torch.isfinite(C[[0, 2, 3]]).all()


@pytest.mark.parametrize("layout", ["row", "col"])
def test_batches_strides_and_unaligned_sources(gm, h, layout):
    x = sample(3 * 40, 70, torch.bfloat16, 4).view(3, 40, 70)
    big = torch.zeros((3, 80, 83), dtype=torch.bfloat16, device="cuda")
    view = big[:, 1:41, 3:73] if layout == "col" else big[:, 1:71, 3:43]
    view.copy_(x if layout == "col" else x.transpose(1, 2))
    q = gm.mx4_empty(120, 70)
    h.mx4_quantise(view, q, layout)
    codes, scales, values = definition(x.reshape(120, 70))
    assert torch.equal(unpack(q)[0], codes) and torch.equal(unpack(q)[1], scales)
    out = torch.zeros((120, 75), dtype=torch.bfloat16, device="cuda")
    h.mx4_dequantise(q, out[:, 2:72])
    h.sync_status()
    assert torch.equal(out[:, 2:72].cpu().double(), values) and (out[:, :2] == 0).all() and (out[:, 72:] == 0).all()


def operands(gm, h, M, N, K, seed):
    a, b = sample(M, K, torch.float32, seed), sample(N, K, torch.float32, seed + 1)
    aq, bq = quantise(gm, h, a), quantise(gm, h, b)
    va, vb = torch.empty((M, K), device="cuda"), torch.empty((N, K), device="cuda")
    h.mx4_dequantise(aq, va)
    h.mx4_dequantise(bq, vb)
    return aq, bq, va.cpu().double(), vb.cpu().double()


def assert_close(C, ref, S, K):
    assert C.dtype == torch.float32
    tol = (K + 2) * 2.0 ** -23 * S
    err = (C.cpu().double() - ref).abs()
    over = ~(err <= tol)
    assert not over.any(), f"{int(over.sum())} elements off, worst {float((err / (S + 1e-300)).max()):.3e} of S"


@pytest.mark.parametrize("shape", [(1, 1, 1), (1, 300, 64), (5, 130, 31), (33, 129, 1000), (130, 260, 513),
                                   (300, 520, 256), (17, 4096, 96), (257, 511, 1536)])
def test_product(gm, h, shape):
    M, N, K = shape
    aq, bq, a, b = operands(gm, h, M, N, K, 5)
    C = torch.full((M, N), float("nan"), device="cuda")
    h.run_mx4(aq, bq, C)
    h.sync_status()
    assert_close(C, a @ b.T, a.abs() @ b.abs().T, K)
    half = torch.full_like(C, float("nan"), dtype=torch.bfloat16)
    h.run_mx4(aq, bq, half)
    h.sync_status()
    assert torch.equal(half, C.bfloat16())


@pytest.mark.parametrize("tile", [1032, 1064, 1128, 1224, 1256, 2032, 2064, 2128, 2224, 21032, 41128, 81064])
@pytest.mark.parametrize("K", [200, 2080, 5000])
def test_every_tile(gm, h, tile, K):
    """Tiles enough for several accumulator hand-overs a CTA."""
    h.set_option(gm.GEMM_OPT_GROUPED_TILE, tile)
    h.set_option(gm.GEMM_OPT_MAX_CTAS, 4)
    M, N = 700, 1000
    aq, bq, a, b = operands(gm, h, M, N, K, 7)
    C = torch.full((M, N), float("nan"), device="cuda")
    h.run_mx4(aq, bq, C)
    h.sync_status()
    assert_close(C, a @ b.T, a.abs() @ b.abs().T, K)


@pytest.mark.parametrize("tile", [0, 1032, 1256, 2064, 2256, 21032, 81128])
@pytest.mark.parametrize("sizes", [[1], [0, 3, 0, 0, 40], [300, 0, 17, 128, 257, 1], [(5 * i) % 7 for i in range(90)]],
                         ids=lambda s: f"{len(s)}groups")
def test_grouped_product(gm, h, sizes, tile):
    h.set_option(gm.GEMM_OPT_GROUPED_TILE, tile)
    G, rows, N, K = len(sizes), sum(sizes) + 4, 150, 330
    bounds = [2]
    for s in sizes:
        bounds.append(bounds[-1] + s)
    aq, bq, a, b = operands(gm, h, rows, G * N, K, 9)
    C = torch.full((rows, N), 7.0, device="cuda")
    h.run_mx4_grouped(aq, bq, torch.tensor(bounds, device="cuda"), C)
    h.sync_status()
    for g in range(G):
        lo, hi = bounds[g], bounds[g + 1]
        w = b[g * N:(g + 1) * N]
        assert_close(C[lo:hi], a[lo:hi] @ w.T, a[lo:hi].abs() @ w.abs().T, K)
    assert (C[:2] == 7).all() and (C[bounds[-1]:] == 7).all()


def test_scales_of_every_magnitude(gm, h):
    """Block exponents from far below to far above 1 whose products stay in FP32."""
    gen = torch.Generator().manual_seed(11)
    K = 512
    ea = torch.randint(-50, 50, (24, K // 32), generator=gen).float()
    a = torch.randn((24, K), generator=gen) * torch.exp2(ea).repeat_interleave(32, 1)
    b = torch.randn((140, K), generator=gen) * torch.exp2(torch.randint(-50, 50, (140, 1), generator=gen).float())
    aq, bq = quantise(gm, h, a), quantise(gm, h, b)
    va, vb = definition(a)[2], definition(b)[2]
    C = torch.empty((24, 140), device="cuda")
    h.run_mx4(aq, bq, C)
    h.sync_status()
    assert_close(C, va @ vb.T, va.abs() @ vb.abs().T, K)


def test_empty_sums_and_empty_calls(gm, h):
    C = torch.full((3, 5), 7.0, device="cuda")
    z = lambda n: gm.Mx4(torch.empty((n, 16), dtype=torch.uint8, device="cuda"),
                         torch.empty((n, 16), dtype=torch.uint8, device="cuda"), 0)
    h.run_mx4(z(3), z(5), C)
    h.sync_status()
    assert (C == 0).all()
    h.run_mx4(gm.mx4_empty(0, 64), gm.mx4_empty(5, 64), C[:0])
    assert h.last_path == "noop"


def test_expired_wait_is_reported_and_the_handle_recovers(gm, h):
    M, N, K = 300, 520, 1024
    aq, bq, a, b = operands(gm, h, M, N, K, 13)
    C = torch.zeros((M, N), device="cuda")
    h.set_option(gm.GEMM_OPT_WAIT_TIMEOUT_NS, 20_000_000)
    for tile in (1064, 2256, 41064):
        h.set_option(gm.GEMM_OPT_GROUPED_TILE, tile)
        h.set_option(gm.GEMM_OPT_DEBUG_DROP_LOAD, 1)
        h.run_mx4(aq, bq, C)
        with pytest.raises(gm.GemmError) as e:
            h.sync_status()
        assert e.value.code == gm.GEMM_ERR_TIMEOUT
        h.set_option(gm.GEMM_OPT_DEBUG_DROP_LOAD, 0)
        h.run_mx4(aq, bq, C)
        h.sync_status()
        assert_close(C, a @ b.T, a.abs() @ b.abs().T, K)


def test_wrong_tensors_are_refused(gm, h):
    q, C = gm.mx4_empty(4, 64), torch.zeros(4, 4, device="cuda")
    x = torch.zeros(4, 64, device="cuda")
    for call in (lambda: h.mx4_quantise(x[:, :32], q), lambda: h.mx4_quantise(x.half(), q),
                 lambda: h.mx4_quantise(x.cpu(), q), lambda: h.mx4_dequantise(q, x[:3]),
                 lambda: h.run_mx4(q, gm.mx4_empty(4, 96), C), lambda: h.run_mx4(q, q, C[:, :3]),
                 lambda: h.run_mx4_grouped(q, q, torch.tensor([0, 1, 4], device="cuda"), C)):
        with pytest.raises(ValueError):
            call()
    odd = gm.Mx4(torch.zeros((4, 40), dtype=torch.uint8, device="cuda"), q.scales, 64)  # a pitch of 40 bytes
    with pytest.raises(gm.GemmError) as e:
        h.run_mx4(odd, q, C)
    assert e.value.code == gm.GEMM_ERR_ALIGNMENT
