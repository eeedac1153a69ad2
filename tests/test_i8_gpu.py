"""8-bit integer products on the GPU: quantisation bit for bit against its
definition in FP64, products against integer sums.

A sum of products of codes that fits 24 bits is exact, so the FP32 result is
(sum * row scale) * column scale, two FP32 roundings, bit for bit, and the BF16
result that value rounded once.  Longer sums in FP32 add parts of 768 products,
at most 2^24 each, with one rounding of the running sum a part: parts * 2^-24
of the sum of the parts' sizes, and the two roundings of the scales.
"""
import math

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


def definition(x):
    """(codes as int64, scales as float32) of a 2-D tensor."""
    x = x.double()
    fine = torch.isfinite(x).all(1)
    top = torch.where(fine, torch.nan_to_num(x).abs().amax(1), math.nan)
    scales = (top / 127).float()
    v = x / scales.double()[:, None]
    codes = torch.where((scales > 0)[:, None], torch.round(v).clamp(-127, 127), torch.zeros_like(v))
    return codes.long(), scales


def same(a, b):
    return torch.equal(torch.nan_to_num(a, nan=-7.0), torch.nan_to_num(b, nan=-7.0))


def quantise(gm, h, x, layout="col"):
    rows, K = x.shape
    q = gm.i8_empty(rows, K)
    q.codes.fill_(99)
    q.scales.fill_(-9)
    h.i8_quantise((x if layout == "col" else x.t().contiguous()).cuda(), q, layout)
    return q


def sample(rows, K, dtype, seed):
    """Normal values, each row at a scale of its own."""
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, K), generator=gen)
    return (x * torch.exp2(torch.randint(-20, 20, (rows, 1), generator=gen).float())).to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["row", "col"])
@pytest.mark.parametrize("shape", [(1, 1), (3, 7), (9, 8), (2, 33), (40, 100), (33, 256), (5, 257), (70, 1000),
                                   (9, 1024), (3, 1031), (2, 4096), (3, 4100), (2, 16384), (2, 20007), (1300, 24)])
def test_quantise_matches_the_definition(gm, h, shape, layout, dtype):
    x = sample(*shape, dtype, 1)
    q = quantise(gm, h, x, layout)
    codes, scales = definition(x)
    assert torch.equal(q.scales.cpu(), scales)
    assert torch.equal(q.codes[:, :shape[1]].cpu().long(), codes)
    assert (q.codes[:, shape[1]:] == 99).all()
    out = torch.empty(shape, dtype=dtype, device="cuda")
    h.i8_dequantise(q, out)
    h.sync_status()
    assert torch.equal(out.cpu(), (codes.float() * scales[:, None]).to(dtype))


@pytest.mark.parametrize("layout", ["row", "col"])
def test_ties_and_small_scales(gm, h, layout):
    gen = torch.Generator().manual_seed(2)
    x = torch.zeros(9, 64)
    x[0, :6] = torch.tensor([127.0, 0.5, 1.5, -2.5, 126.5, -0.5])      # scale 1: ties to even
    x[1, :6] = torch.nextafter(x[0, :6], torch.tensor(1e9))            # a hair above
    x[2, :6] = torch.nextafter(x[0, :6], torch.tensor(-1e9))           # a hair below
    x[2, 0] = x[1, 0] = 127.0
    x[3] = torch.randint(-200, 200, (64,), generator=gen) * 2.0 ** -149  # subnormal
    x[4, :3] = torch.tensor([2.0 ** -149, -(2.0 ** -149), 0.0])          # the scale rounds to zero
    x[5] = torch.randn(64, generator=gen) * 1e-36
    x[6, :3] = torch.tensor([3.4e38, -3.4e38, 1e38])
    x[7, :2] = torch.tensor([100.0, 50.0])
    s = float(torch.tensor(100.0) / 127)  # halves of the scale, in FP32
    x[7, 2:34] = torch.arange(32) * s + s / 2
    q = quantise(gm, h, x, layout)
    codes, scales = definition(x)
    assert torch.equal(q.scales.cpu(), scales) and torch.equal(q.codes[:, :64].cpu().long(), codes)
    assert codes[0, :6].tolist() == [127, 0, 2, -2, 126, 0] and (codes[8] == 0).all() and scales[8] == 0


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_a_row_that_is_not_finite_becomes_nan(gm, h, bad):
    x = sample(4, 300, torch.float32, 3)
    x[1, 40] = bad
    for layout in ("col", "row"):
        q = quantise(gm, h, x, layout)
        codes, scales = definition(x)
        assert same(q.scales.cpu(), scales) and torch.isnan(scales).tolist() == [False, True, False, False]
        assert torch.equal(q.codes[:, :300].cpu().long(), codes)
        B = quantise(gm, h, sample(130, 300, torch.float32, 4))
        C, D = torch.empty((4, 130), device="cuda"), torch.empty((130, 4), device="cuda")
        h.run_i8(q, B, C)
        h.run_i8(B, q, D)
        h.sync_status()
        assert torch.isnan(C[1]).all() and torch.isfinite(C[[0, 2, 3]]).all()
        assert torch.isnan(D[:, 1]).all() and torch.isfinite(D[:, [0, 2, 3]]).all()


@pytest.mark.parametrize("layout", ["row", "col"])
def test_batches_strides_and_unaligned_sources(gm, h, layout):
    x = sample(3 * 40, 70, torch.bfloat16, 5).view(3, 40, 70)
    big = torch.zeros((3, 80, 83), dtype=torch.bfloat16, device="cuda")
    view = big[:, 1:41, 3:73] if layout == "col" else big[:, 1:71, 3:43]
    view.copy_(x if layout == "col" else x.transpose(1, 2))
    q = gm.i8_empty(120, 70)
    h.i8_quantise(view, q, layout)
    codes, scales = definition(x.reshape(120, 70))
    assert torch.equal(q.scales.cpu(), scales) and torch.equal(q.codes[:, :70].cpu().long(), codes)
    out = torch.zeros((120, 75), dtype=torch.bfloat16, device="cuda")
    h.i8_dequantise(q, out[:, 2:72])
    h.sync_status()
    assert torch.equal(out[:, 2:72].cpu(), (codes.float() * scales[:, None]).bfloat16())
    assert (out[:, :2] == 0).all() and (out[:, 72:] == 0).all()


def operand(gm, rows, K, seed, pad=0, low=-128):
    """Random codes and scales, the padding bytes set to junk."""
    gen = torch.Generator().manual_seed(seed)
    pitch = gm.gemm_i8_code_pitch(K) + 16 * pad
    codes = torch.randint(-128, 128, (rows, pitch), generator=gen).to(torch.int8)
    codes[:, :K] = codes[:, :K].clamp(min=low)
    scales = torch.rand(rows, generator=gen) + 0.5
    return gm.I8(codes.cuda(), scales.cuda(), K), codes[:, :K].long(), scales


def product(a, b):
    """Integer sums (FP64 holds them exactly up to 2^53)."""
    return (a.double() @ b.double().T).long()


def expected(sums, sa, sb):
    return (sums.float() * sa[:, None]) * sb


@pytest.mark.parametrize("shape", [(1, 1, 1), (1, 300, 64), (5, 130, 31), (33, 129, 1000), (130, 260, 513),
                                   (300, 520, 256), (17, 4096, 96), (257, 511, 768), (2000, 4100, 128)])
def test_product(gm, h, shape):
    M, N, K = shape
    A, a, sa = operand(gm, M, K, 5)
    B, b, sb = operand(gm, N, K, 6, pad=1)
    sums = product(a, b)
    assert sums.abs().max() <= 2 ** 24
    C = torch.full((M, N), float("nan"), device="cuda")
    h.run_i8(A, B, C)
    h.sync_status()
    assert torch.equal(C.cpu(), expected(sums, sa, sb))
    half = torch.full_like(C, float("nan"), dtype=torch.bfloat16)
    h.run_i8(A, B, half)
    h.sync_status()
    assert torch.equal(half.cpu(), expected(sums, sa, sb).bfloat16())


TILES = [1032, 1064, 1128, 2032, 2064, 2128, 2224, 2256, 21032, 41128, 81064]


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("K", [200, 1030, 5000])
def test_every_tile(gm, h, tile, K, out):
    """Several tiles a CTA; random codes, whose sums stay within 24 bits."""
    h.set_option(gm.GEMM_OPT_GROUPED_TILE, tile)
    h.set_option(gm.GEMM_OPT_MAX_CTAS, 4)
    M, N = 700, 1000
    A, a, sa = operand(gm, M, K, 7)
    B, b, sb = operand(gm, N, K, 8)
    sums = product(a, b)
    assert sums.abs().max() < 2 ** 24
    C = torch.full((M, N + 3), 7.0, dtype=out, device="cuda")
    h.run_i8(A, B, C[:, 1:N + 1])
    h.sync_status()
    assert torch.equal(C[:, 1:N + 1].cpu(), expected(sums, sa, sb).to(out))
    assert (C[:, 0] == 7).all() and (C[:, N + 1:] == 7).all()


@pytest.mark.parametrize("tile", [0] + TILES)
def test_largest_sums(gm, h, tile):
    """All products 2^14, or all -127 * 128: exact at K = 1024; at K = 20000 the
    FP32 result within a rounding a part, the BF16 one within its own rounding
    and the accumulator's loss of 2^-23 of the sum for every 16 products."""
    h.set_option(gm.GEMM_OPT_GROUPED_TILE, tile)
    M, N = 70, 150
    for K in (1024, 20000):
        A, a, sa = operand(gm, M, K, 9)
        B, b, sb = operand(gm, N, K, 10)
        for code in (-128, 127):
            A.codes.fill_(code)
            B.codes.fill_(-128)
            total = K * code * -128
            ref = total * sa.double()[:, None] * sb.double()
            C = torch.empty((M, N), device="cuda")
            half = torch.empty((M, N), device="cuda", dtype=torch.bfloat16)
            h.run_i8(A, B, C)
            h.run_i8(A, B, half)
            h.sync_status()
            parts = math.ceil(K / 768) if K > 1024 else 0
            assert ((C.cpu().double() - ref).abs() <= (parts + 2) * 2.0 ** -24 * ref.abs()).all()
            loss = max(0, K - 1024) / 16 * 2.0 ** -23
            assert ((half.cpu().double() - ref).abs() <= (2.0 ** -8 + loss + 2.0 ** -22) * ref.abs()).all()


@pytest.mark.parametrize("tile", [0, 1032, 1128, 2064, 2256, 21032, 81128])
@pytest.mark.parametrize("sizes", [[1], [0, 3, 0, 0, 40], [300, 0, 17, 128, 257, 1], [(5 * i) % 7 for i in range(90)]],
                         ids=lambda s: f"{len(s)}groups")
def test_grouped_product(gm, h, sizes, tile):
    h.set_option(gm.GEMM_OPT_GROUPED_TILE, tile)
    G, rows, N, K = len(sizes), sum(sizes) + 4, 150, 330
    bounds = [2]
    for s in sizes:
        bounds.append(bounds[-1] + s)
    A, a, sa = operand(gm, rows, K, 11)
    B, b, sb = operand(gm, G * N, K, 12)
    for out in (torch.float32, torch.bfloat16):
        C = torch.full((rows, N), 7.0, device="cuda", dtype=out)
        h.run_i8_grouped(A, B, torch.tensor(bounds, device="cuda"), C)
        h.sync_status()
        got = C.cpu()
        for g in range(G):
            lo, hi = bounds[g], bounds[g + 1]
            w = slice(g * N, (g + 1) * N)
            assert torch.equal(got[lo:hi], expected(product(a[lo:hi], b[w]), sa[lo:hi], sb[w]).to(out))
        assert (got[:2] == 7).all() and (got[bounds[-1]:] == 7).all()


@pytest.mark.parametrize("M,N", [(4, 2048), (64, 2048), (700, 3000), (5000, 8192)])
def test_chosen_tiles(gm, h, M, N):
    A, a, sa = operand(gm, M, 1024, 13)
    B, b, sb = operand(gm, N, 1024, 14)
    some = torch.arange(0, M, max(1, M // 64))
    want = expected(product(a[some], b), sa[some], sb)
    for out in (torch.float32, torch.bfloat16):
        C = torch.empty((M, N), device="cuda", dtype=out)
        h.run_i8(A, B, C)
        h.sync_status()
        assert torch.equal(C[some].cpu(), want.to(out))


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 33, 15), (2, 100, 17), (3, 31, 496), (4, 130, 512), (5, 257, 1000),
                                   (7, 64, 2100), (8, 300, 4096), (1, 40, 11000), (4, 77, 24000), (8, 5000, 130)])
def test_few_rows(gm, h, M, N, K, out):
    A, a, sa = operand(gm, M, K, 31)
    B, b, sb = operand(gm, N, K, 32, pad=1)
    sums = product(a, b)
    assert sums.abs().max() < 2 ** 24
    C = torch.full((M + 2, N + 3), 7.0, device="cuda", dtype=out)
    h.run_i8(A, B, C[1:M + 1, 2:N + 2])
    h.sync_status()
    assert h.last_path == ("i8_rows" if K < 13000 or M <= 4 else h.last_path)
    assert torch.equal(C[1:M + 1, 2:N + 2].cpu(), expected(sums, sa, sb).to(out))
    assert (C[0] == 7).all() and (C[M + 1] == 7).all() and (C[:, :2] == 7).all() and (C[:, N + 2:] == 7).all()


@pytest.mark.parametrize("sizes", [[1] * 40, [0, 3, 0, 9, 1, 20, 0], [17, 0, 0, 0, 0, 0], [0, 0, 0], [8, 8, 1]],
                         ids=lambda s: f"{len(s)}groups{sum(s)}rows")
def test_few_rows_grouped(gm, h, sizes):
    """Groups of many rows among them: they are taken four at a time.  Empty groups
    behind make the groups' average small."""
    rows, N, K = sum(sizes) + 3, 70, 330
    sizes = sizes + [0] * max(0, (rows + 1) // 2 - len(sizes))
    G = len(sizes)
    bounds = [2]
    for s in sizes:
        bounds.append(bounds[-1] + s)
    A, a, sa = operand(gm, rows, K, 33)
    B, b, sb = operand(gm, G * N, K, 34)
    C = torch.full((rows, N), 7.0, device="cuda")
    h.run_i8_grouped(A, B, torch.tensor(bounds, device="cuda"), C)
    h.sync_status()
    assert h.last_path == "grouped_i8_rows"
    for g in range(G):
        lo, hi = bounds[g], bounds[g + 1]
        w = slice(g * N, (g + 1) * N)
        assert torch.equal(C[lo:hi].cpu(), expected(product(a[lo:hi], b[w]), sa[lo:hi], sb[w]))
    assert (C[:2] == 7).all() and (C[bounds[-1]:] == 7).all()
    for bad in ([0, 3, 2] + [rows] * (G - 2), [-1] * G + [2], [0] * G + [rows + 1]):
        C.fill_(7.0)
        h.run_i8_grouped(A, B, torch.tensor(bad, device="cuda"), C)
        with pytest.raises(gm.GemmError) as e:
            h.sync_status()
        assert e.value.code == gm.GEMM_ERR_INVALID and (C == 7).all()


@pytest.mark.parametrize("rows,K", [(4, 24576), (8, 12288)])
def test_few_rows_largest_sums(gm, h, rows, K):
    """Products of 2^14 as long as the kernel takes them, and one off: sums past 24
    bits, rounded once to FP32."""
    A, a, sa = operand(gm, rows, K, 35)
    B, b, sb = operand(gm, 9, K, 36)
    A.codes.fill_(-128)
    B.codes.fill_(-128)
    B.codes[:, 5] = 1
    C = torch.empty((rows, 9), device="cuda")
    h.run_i8(A, B, C)
    h.sync_status()
    assert h.last_path == "i8_rows"
    assert torch.equal(C.cpu(), expected(torch.full((rows, 9), (K - 1) * 2 ** 14 - 128), sa, sb))


@pytest.mark.parametrize("rows,groups", [(1536, 768), (1537, 769), (1, 1024), (300, 150)])
def test_few_rows_most_passes(gm, h, rows, groups):
    """A pass for every row, and every row in one group."""
    N, K = 9, 40
    A, a, sa = operand(gm, rows, K, 37)
    B, b, sb = operand(gm, groups * N, K, 38)
    for bounds in ([min(rows, g) for g in range(groups)] + [rows], [0] * (groups // 2) + [rows] * (groups - groups // 2 + 1)):
        C = torch.full((rows, N), 7.0, device="cuda")
        h.run_i8_grouped(A, B, torch.tensor(bounds, device="cuda"), C)
        h.sync_status()
        assert (h.last_path == "grouped_i8_rows") == (rows <= 1536)
        for g in range(groups):
            lo, hi = bounds[g], bounds[g + 1]
            w = slice(g * N, (g + 1) * N)
            if hi > lo:
                assert torch.equal(C[lo:hi].cpu(), expected(product(a[lo:hi], b[w]), sa[lo:hi], sb[w]))


def test_empty_sums_and_empty_calls(gm, h):
    C = torch.full((3, 5), 7.0, device="cuda")
    z = lambda n: gm.I8(torch.empty((n, 16), dtype=torch.int8, device="cuda"),
                        torch.full((n,), math.nan, device="cuda"), 0)
    h.run_i8(z(3), z(5), C)
    h.sync_status()
    assert (C == 0).all()
    h.run_i8(gm.i8_empty(0, 64), gm.i8_empty(5, 64), C[:0])
    assert h.last_path == "noop"


@pytest.mark.parametrize("tile", [1064, 2256, 41064])
def test_refused_offsets(gm, h, tile):
    h.set_option(gm.GEMM_OPT_GROUPED_TILE, tile)
    A, a, sa = operand(gm, 300, 512, 15)
    B, b, sb = operand(gm, 3 * 100, 512, 16)
    for bad in ([0, 5, 3, 300], [-1, 2, 3, 300], [0, 2, 3, 301]):
        C = torch.full((300, 100), 7.0, device="cuda")
        h.run_i8_grouped(A, B, torch.tensor(bad, device="cuda"), C)
        with pytest.raises(gm.GemmError) as e:
            h.sync_status()
        assert e.value.code == gm.GEMM_ERR_INVALID and (C == 7).all()


def test_expired_wait_is_reported_and_the_handle_recovers(gm, h):
    M, N, K = 300, 520, 1000
    A, a, sa = operand(gm, M, K, 17)
    B, b, sb = operand(gm, N, K, 18)
    ref = expected(product(a, b), sa, sb)
    C = torch.zeros((M, N), device="cuda")
    h.set_option(gm.GEMM_OPT_WAIT_TIMEOUT_NS, 20_000_000)
    for tile in (1064, 2256, 41064):
        h.set_option(gm.GEMM_OPT_GROUPED_TILE, tile)
        h.set_option(gm.GEMM_OPT_DEBUG_DROP_LOAD, 1)
        h.run_i8(A, B, C)
        with pytest.raises(gm.GemmError) as e:
            h.sync_status()
        assert e.value.code == gm.GEMM_ERR_TIMEOUT
        h.set_option(gm.GEMM_OPT_DEBUG_DROP_LOAD, 0)
        h.run_i8(A, B, C)
        h.sync_status()
        assert torch.equal(C.cpu(), ref)


def test_streams_and_captured_graphs(gm, h):
    """Calls that convert in the workspace take turns on several streams; a captured
    quantisation and product replays on new activations, its first call included."""
    M, N, K = 3000, 1024, 512
    h.set_option(gm.GEMM_OPT_GROUPED_TILE, 2256)
    B, b, sb = operand(gm, N, K, 19)
    sets = [operand(gm, M, K, 20 + i) for i in range(3)]
    refs = [expected(product(a, b), sa, sb) for _, a, sa in sets]
    outs = [torch.empty((M, N), device="cuda") for _ in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(4):
        for (A, _, _), C, s in zip(sets, outs, streams):
            h.run_i8(A, B, C, stream=s)
    torch.cuda.synchronize()
    for C, ref in zip(outs, refs):
        assert torch.equal(C.cpu(), ref)
    with gm.Gemm(0) as fresh:
        x = torch.zeros((M, K), device="cuda", dtype=torch.bfloat16)
        q, C = gm.i8_empty(M, K), torch.empty((M, N), device="cuda")
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            fresh.i8_quantise(x, q)
            fresh.run_i8(q, B, C)
        for seed in (1, 2):
            new = sample(M, K, torch.bfloat16, seed)
            x.copy_(new)
            graph.replay()
            torch.cuda.synchronize()
            codes, scales = definition(new)
            assert torch.equal(C.cpu(), expected(product(codes, b), scales, sb))


def test_wrong_tensors_are_refused(gm, h):
    q, C = gm.i8_empty(4, 64), torch.zeros(4, 4, device="cuda")
    x = torch.zeros(4, 64, device="cuda")
    for call in (lambda: h.i8_quantise(x[:, :32], q), lambda: h.i8_quantise(x.half(), q),
                 lambda: h.i8_quantise(x.cpu(), q), lambda: h.i8_dequantise(q, x[:3]),
                 lambda: h.run_i8(q, gm.i8_empty(4, 96), C), lambda: h.run_i8(q, q, C[:, :3]),
                 lambda: h.run_i8(q, gm.i8_empty(4, 64, device="cpu"), C),
                 lambda: h.run_i8_grouped(q, q, torch.tensor([0, 1, 4], device="cuda"), C)):
        with pytest.raises(ValueError):
            call()
    odd = gm.I8(torch.zeros((4, 72), dtype=torch.int8, device="cuda"), q.scales, 64)  # a pitch of 72 bytes
    with pytest.raises(gm.GemmError) as e:
        h.run_i8(odd, q, C)
    assert e.value.code == gm.GEMM_ERR_ALIGNMENT


def test_routed_quantised_expert_layer(gm, h):
    """Router, quantisation and grouped product one behind the other."""
    from dense_gemm_sm100_gb300.experts import route
    gen = torch.Generator().manual_seed(30)
    T, E, k, K, N = 100, 10, 2, 256, 136
    r = route(torch.randn((T, E), generator=gen).cuda(), k, handle=h)
    x = torch.randn((T, K), generator=gen).bfloat16().cuda()
    W = quantise(gm, h, torch.randn((E * N, K), generator=gen))
    rows = x[r.order // k]
    q = gm.i8_empty(T * k, K)
    h.i8_quantise(rows, q)
    y = torch.empty((T * k, N), device="cuda")
    h.run_i8_grouped(q, W, r.offsets, y)
    h.sync_status()
    codes, scales = definition(rows.cpu())
    wc, ws = W.codes[:, :K].cpu().long(), W.scales.cpu()
    b = r.offsets.tolist()
    for g in range(E):
        w = slice(g * N, (g + 1) * N)
        rows_g = slice(b[g], b[g + 1])
        assert torch.equal(y[rows_g].cpu(), expected(product(codes[rows_g], wc[w]), scales[rows_g], ws[w]))
