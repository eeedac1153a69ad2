"""Grouped expert products and their gradients on the GPU, element by element
against FP64.

Bounds, with S = sum |a b| of an element over K terms: BF16 products are exact
in FP32 and each of the K additions loses less than 2^-23 of the partial sum,
so |C - ref| <= (K + 2) 2^-23 S; a BF16 result is the FP32 result of the same
call rounded once, bit for bit, unless FP32 results are summed in segments
(more than 12 stages of 64 elements), and then within half a unit of its eight
significant bits, 2^-8 |C|, of a sum within that bound; TF32 keeps 11 significant bits of each operand by
dropping the rest, less than 2^-10 each and so 2^-9 of a product, framed as
2^-9 + 2^-20.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

# CTAs and rows of a tile; 10000 S: the contraction over clusters of S CTAs
TILES = [1032, 1064, 1128, 1256, 2032, 2064, 2128, 2256, 21032, 41064, 81032, 81128]


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


def bounds_of(sizes, start=0):
    b = [start]
    for s in sizes:
        b.append(b[-1] + s)
    return b


def device_offsets(b):
    return torch.tensor(b, dtype=torch.int64, device="cuda")


def draw(shape, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=gen).to(torch.bfloat16 if dtype == "bf16" else torch.float32)


def tolerance(S, K, dtype):
    t = (K + 2) * 2.0 ** -23 * S
    return t + (2.0 ** -9 + 2.0 ** -20) * S if dtype == "tf32" else t


def assert_close(C, ref, S, K, dtype):
    assert C.dtype == torch.float32
    err = (C.cpu().double() - ref).abs()
    over = ~(err <= tolerance(S, K, dtype))
    assert not over.any(), f"{int(over.sum())} elements off, worst {float((err / (S + 1e-300)).max()):.3e} of S"


def forward_ref(A, W, b):
    """W logical (groups, K, N)."""
    A, W = A.double(), W.double()
    spans = [(g, b[g], b[g + 1]) for g in range(W.shape[0])]
    ref = torch.zeros(A.shape[0], W.shape[2], dtype=torch.float64)
    S = torch.zeros_like(ref)
    for g, lo, hi in spans:
        ref[lo:hi] = A[lo:hi] @ W[g]
        S[lo:hi] = A[lo:hi].abs() @ W[g].abs()
    return ref, S


def wgrad_ref(A, B, b):
    A, B = A.double(), B.double()
    G = len(b) - 1
    ref = torch.stack([A[b[g]:b[g + 1]].T @ B[b[g]:b[g + 1]] for g in range(G)])
    S = torch.stack([A[b[g]:b[g + 1]].abs().T @ B[b[g]:b[g + 1]].abs() for g in range(G)])
    return ref, S


def run_forward(h, A, W, b, layout, dtype, out=torch.float32):
    B = (W if layout == "row" else W.transpose(1, 2)).contiguous().cuda()
    C = torch.full((A.shape[0], W.shape[2]), float("nan"), dtype=out, device="cuda")
    h.run_grouped(A.cuda(), B, device_offsets(b), C, layout, dtype)
    h.sync_status()
    return C


SIZES = [
    [1], [33], [0, 0, 5, 0], [257, 0, 31, 64, 1, 2, 0, 130],
    [(7 * i * i) % 23 for i in range(200)],  # many groups, a fifth of them short
]


@pytest.mark.parametrize("layout", ["row", "col"])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}groups")
@pytest.mark.parametrize("KN", [(64, 128), (200, 328), (1000, 64)])
def test_bf16_sizes(h, sizes, KN, layout):
    K, N = KN
    b = bounds_of(sizes)
    A, W = draw((b[-1], K), "bf16", 1), draw((len(sizes), K, N), "bf16", 2)
    C = run_forward(h, A, W, b, layout, "bf16")
    assert_close(C, *forward_ref(A, W, b), K, "bf16")
    half = run_forward(h, A, W, b, layout, "bf16", torch.bfloat16)
    if K <= 12 * 64:
        assert torch.equal(half, C.bfloat16())
    else:
        ref, S = forward_ref(A, W, b)
        t = tolerance(S, K, "bf16")
        assert ((half.cpu().double() - ref).abs() <= t + 2.0 ** -8 * (ref.abs() + t)).all()


@pytest.mark.parametrize("layout", ["row", "col"])
@pytest.mark.parametrize("dtype", ["bf16", "tf32"])
@pytest.mark.parametrize("KN", [(1, 1), (7, 5), (65, 129), (100, 130), (333, 127)])
def test_odd_sizes_are_repacked(h, KN, dtype, layout):
    K, N = KN
    b = bounds_of([3, 0, 70, 1])
    A, W = draw((b[-1], K), dtype, 3), draw((4, K, N), dtype, 4)
    assert_close(run_forward(h, A, W, b, layout, dtype), *forward_ref(A, W, b), K, dtype)


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("layout", ["row", "col"])
@pytest.mark.parametrize("dtype", ["bf16", "tf32"])
def test_every_tile(h, gm, dtype, layout, tile):
    h.set_option(gm.GEMM_OPT_GROUPED_TILE, tile)
    b = bounds_of([300, 0, 17, 128, 257, 1])
    K, N = 264, 392
    A, W = draw((b[-1], K), dtype, 5), draw((6, K, N), dtype, 6)
    assert_close(run_forward(h, A, W, b, layout, dtype), *forward_ref(A, W, b), K, dtype)
    assert f"x{tile % 1000}" in h.last_path and (f"+splitk{tile // 10000}" in h.last_path) == (tile > 9999)


@pytest.mark.parametrize("tile", [0, 1128, 1256, 2128, 2256, 21128, 81128])
@pytest.mark.parametrize("dtype", ["bf16", "tf32"])
@pytest.mark.parametrize("MN", [(1, 1), (72, 40), (256, 128), (200, 333), (129, 520)])
def test_wgrad(h, gm, MN, dtype, tile):
    h.set_option(gm.GEMM_OPT_GROUPED_TILE, tile)
    M, N = MN
    sizes = [300, 0, 17, 64, 1, 0, 131]
    b = bounds_of(sizes)
    A, B = draw((b[-1], M), dtype, 7), draw((b[-1], N), dtype, 8)
    C = torch.full((len(sizes), M, N), float("nan"), device="cuda")
    h.run_grouped_wgrad(A.cuda(), B.cuda(), device_offsets(b), C, dtype)
    h.sync_status()
    assert_close(C, *wgrad_ref(A, B, b), max(sizes), dtype)
    assert torch.equal(C[1], torch.zeros_like(C[1]))  # a group without rows
    if dtype == "bf16":
        half = torch.full_like(C, float("nan"), dtype=torch.bfloat16)
        h.run_grouped_wgrad(A.cuda(), B.cuda(), device_offsets(b), half, dtype)
        h.sync_status()
        assert torch.equal(half, C.bfloat16())


@pytest.mark.parametrize("dtype", ["bf16", "tf32"])
def test_integers_are_exact(h, dtype):
    gen = torch.Generator().manual_seed(9)
    b = bounds_of([40, 0, 300, 3])
    d = torch.bfloat16 if dtype == "bf16" else torch.float32
    A = torch.randint(-8, 9, (b[-1], 136), generator=gen).to(d)
    W = torch.randint(-8, 9, (4, 136, 200), generator=gen).to(d)
    assert torch.equal(run_forward(h, A, W, b, "row", dtype).cpu().double(), forward_ref(A, W, b)[0])
    dY = torch.randint(-8, 9, (b[-1], 200), generator=gen).to(d)
    C = torch.empty((4, 136, 200), device="cuda")
    h.run_grouped_wgrad(A.cuda(), dY.cuda(), device_offsets(b), C, dtype)
    assert torch.equal(C.cpu().double(), wgrad_ref(A, dY, b)[0])


@pytest.mark.parametrize("rows", [1, 7, 40, 300])
@pytest.mark.parametrize("dtype", ["bf16", "tf32"])
def test_few_tiles_and_a_long_contraction_are_cut(h, gm, dtype, rows):
    """Fewer tiles than SMs: clusters share K, unless the option forbids it."""
    b = bounds_of([rows])
    K, N = 4104, 200
    A, W = draw((rows, K), dtype, 32), draw((1, K, N), dtype, 33)
    ref = forward_ref(A, W, b)
    cut = run_forward(h, A, W, b, "row", dtype)
    assert "+splitk" in h.last_path
    assert_close(cut, *ref, K, dtype)
    if dtype == "bf16":
        assert torch.equal(run_forward(h, A, W, b, "row", dtype, torch.bfloat16), cut.bfloat16())
    h.set_option(gm.GEMM_OPT_SPLIT_K, 1)
    whole = run_forward(h, A, W, b, "row", dtype)
    assert "+splitk" not in h.last_path
    assert_close(whole, *ref, K, dtype)


@pytest.mark.parametrize("tile", [0, 1064, 1256, 2256])
def test_long_sums_of_one_sign_keep_fp32_accuracy(h, gm, tile):
    """The tensor core drops up to one unit (2^-23) of its FP32 accumulator per
    addition; the library lets at most 48 additions pass between roundings to
    nearest, so results of positive operands stay within 48 2^-23 of the sum at
    any K (512 additions in one go at K = 8192)."""
    h.set_option(gm.GEMM_OPT_GROUPED_TILE, tile)
    gen = torch.Generator().manual_seed(34)
    rows, K, N = 260, 8192, 256
    A = torch.rand((rows, K), generator=gen).bfloat16()
    W = torch.rand((1, K, N), generator=gen).bfloat16()
    ref = forward_ref(A, W, [0, rows])[0]
    C = run_forward(h, A, W, [0, rows], "row", "bf16").cpu().double()
    assert float(((C - ref).abs() / ref).max()) <= 48 * 2.0 ** -23
    g = torch.empty((1, 256, 128), device="cuda")
    A, B = torch.rand((K, 256), generator=gen).bfloat16(), torch.rand((K, 128), generator=gen).bfloat16()
    h.run_grouped_wgrad(A.cuda(), B.cuda(), device_offsets([0, K]), g, "bf16")
    h.sync_status()
    ref = A.double().T @ B.double()
    assert float(((g[0].cpu().double() - ref).abs() / ref).max()) <= 48 * 2.0 ** -23


@pytest.mark.parametrize("tile", [1128, 2256])
@pytest.mark.parametrize("dtype", ["bf16", "tf32"])
def test_a_long_group_among_short_ones_is_summed_as_alone(h, gm, dtype, tile):
    """The length at which a weight gradient is summed in segments is the
    group's own: its bits do not depend on how long the others are."""
    h.set_option(gm.GEMM_OPT_GROUPED_TILE, tile)
    sizes = [3] * 31 + [2100]
    b = bounds_of(sizes)
    A, B = draw((b[-1], 136), dtype, 21).cuda(), draw((b[-1], 264), dtype, 22).cuda()
    C = torch.empty((len(sizes), 136, 264), device="cuda")
    h.run_grouped_wgrad(A, B, device_offsets(b), C, dtype)
    alone = torch.empty((1, 136, 264), device="cuda")
    h.run_grouped_wgrad(A[b[-2]:], B[b[-2]:], device_offsets([0, sizes[-1]]), alone, dtype)
    h.sync_status()
    assert torch.equal(C[-1], alone[0])


def test_rows_outside_the_groups_and_padding_are_untouched(h):
    b = bounds_of([20, 0, 45], start=7)
    rows, K, N = 90, 72, 100
    A, W = draw((rows, 80), "bf16", 10)[:, :K], draw((3, K, N), "bf16", 11)
    store = torch.full((rows, N + 12), -3.0, device="cuda")
    h.run_grouped(draw((rows, 80), "bf16", 10).cuda()[:, :K], W.cuda(), device_offsets(b), store[:, :N], "row", "bf16")
    h.sync_status()
    ref, S = forward_ref(A, W, b)
    assert_close(store[7:72, :N], ref[7:72], S[7:72], K, "bf16")
    assert (store[:, N:] == -3).all() and (store[:7] == -3).all() and (store[72:] == -3).all()


@pytest.mark.parametrize("dtype", ["bf16", "tf32"])
@pytest.mark.parametrize("shift", [1, 4])
def test_strides_and_offsets_of_every_operand(h, dtype, shift):
    """Operands cut out of larger tensors: padded pitches, group strides and
    bases that TMA can (shift 4 x 4 bytes) and cannot address."""
    d = torch.bfloat16 if dtype == "bf16" else torch.float32
    b = bounds_of([9, 70, 0, 33])
    K, N, G = 96, 72, 4
    big_a = draw((b[-1], K + 16), dtype, 12).cuda()
    big_w = draw((G, K + 3, N + 24), dtype, 13).cuda()
    A, W = big_a[:, shift:shift + K], big_w[:, 2:2 + K, shift:shift + N]
    C = torch.zeros((b[-1], N + 5), device="cuda")[:, 3:3 + N]
    h.run_grouped(A, W, device_offsets(b), C, "row", dtype)
    assert_close(C, *forward_ref(A.cpu(), W.cpu(), b), K, dtype)
    dC = draw((b[-1], N + 9), dtype, 14).cuda()[:, shift:shift + N]
    dA = torch.zeros((b[-1], K + 7), device="cuda")[:, 1:1 + K]
    h.run_grouped(dC, W, device_offsets(b), dA, "col", dtype)
    assert_close(dA, *forward_ref(dC.cpu(), W.cpu().transpose(1, 2), b), N, dtype)
    dW = torch.zeros((G, K + 2, N + 6), device="cuda")[:, 1:1 + K, 2:2 + N]
    h.run_grouped_wgrad(A, dC, device_offsets(b), dW, dtype)
    h.sync_status()
    assert_close(dW, *wgrad_ref(A.cpu(), dC.cpu(), b), 70, dtype)
    assert d == A.dtype


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_values_that_are_not_finite_stay_in_their_row_and_group(h, bad):
    b = bounds_of([5, 130, 64, 2])
    K, N = 128, 256
    A, W, dC = draw((b[-1], K), "bf16", 15), draw((4, K, N), "bf16", 16), draw((b[-1], N), "bf16", 17)
    ref, S = forward_ref(A, W, b)
    gref, gS = wgrad_ref(A, dC, b)
    A2 = A.clone()
    A2[5, 3] = bad          # first row of group 1
    A2[134, 100] = bad      # its last row, inside the last stage of the contraction
    C = run_forward(h, A2, W, b, "row", "bf16").cpu()
    keep = torch.ones(b[-1], dtype=torch.bool)
    keep[[5, 134]] = False
    assert_close(C[keep], ref[keep], S[keep], K, "bf16")
    assert not torch.isfinite(C[~keep]).any()
    g = torch.empty((4, K, N), device="cuda")
    h.run_grouped_wgrad(A2.cuda(), dC.cuda(), device_offsets(b), g, "bf16")
    h.sync_status()
    assert_close(g[[0, 2, 3]], gref[[0, 2, 3]], gS[[0, 2, 3]], 64, "bf16")
    assert not torch.isfinite(g[1, 3]).any() and not torch.isfinite(g[1, 100]).any()
    W2 = W.clone()
    W2[2] = bad             # one expert's weights
    C = run_forward(h, A, W2, b, "col", "bf16").cpu()
    assert torch.isfinite(C[:135]).all() and torch.isfinite(C[199:]).all() and not torch.isfinite(C[135:199]).any()


def test_empty_sums_and_empty_calls(h):
    b = device_offsets([2, 2, 5])
    C = torch.full((6, 40), 7.0, device="cuda")
    h.run_grouped(torch.empty((6, 0), device="cuda").bfloat16(), torch.empty((2, 0, 40), device="cuda").bfloat16(), b,
                  C, "row", "bf16")
    h.sync_status()
    assert (C[2:5] == 0).all() and (C[:2] == 7).all() and (C[5:] == 7).all()
    h.run_grouped(torch.empty((0, 16), device="cuda").bfloat16(), torch.empty((2, 16, 40), device="cuda").bfloat16(),
                  device_offsets([0, 0, 0]), C[:0], "row", "bf16")
    assert h.last_path == "noop"
    g = torch.full((2, 16, 40), 7.0, device="cuda")
    h.run_grouped_wgrad(torch.empty((0, 16), device="cuda").bfloat16(), torch.empty((0, 40), device="cuda").bfloat16(),
                        device_offsets([0, 0, 0]), g, "bf16")
    h.sync_status()
    assert (g == 0).all()


@pytest.mark.parametrize("bad", [[0, 5, 3, 8], [-1, 2, 3, 8], [0, 2, 3, 9], [4, 4, 4, 0]])
def test_offsets_that_decrease_or_leave_the_rows_compute_nothing(h, gm, bad):
    A, W = draw((8, 64), "bf16", 18), draw((3, 64, 128), "bf16", 19)
    C = torch.full((8, 128), 7.0, device="cuda")
    h.run_grouped(A.cuda(), W.cuda(), device_offsets(bad), C, "row", "bf16")
    with pytest.raises(gm.GemmError) as e:
        h.sync_status()
    assert e.value.code == gm.GEMM_ERR_INVALID and "offsets" in str(e.value)
    g = torch.full((3, 64, 64), 7.0, device="cuda")
    h.run_grouped_wgrad(A.cuda(), A.cuda(), device_offsets(bad), g, "bf16")
    with pytest.raises(gm.GemmError):
        h.sync_status()
    assert (C == 7).all() and (g == 7).all()
    b = [0, 2, 3, 8]
    assert_close(run_forward(h, A, W, b, "row", "bf16"), *forward_ref(A, W, b), 64, "bf16")


def test_wrong_tensors_are_refused(h):
    A, W = torch.zeros(8, 64, device="cuda").bfloat16(), torch.zeros(3, 64, 128, device="cuda").bfloat16()
    C, o = torch.zeros(8, 128, device="cuda"), device_offsets([0, 1, 2, 8])
    for args in [(A.float(), W, o, C), (A, W.float(), o, C), (A, W, o.int(), C), (A, W, o[:3], C), (A, W, o, C.half()),
                 (A, W, o, C[:, :64]), (A[:, :32], W, o, C), (A.t(), W, o, C), (A.cpu(), W, o, C),
                 (A, W, o.cpu(), C), (A[:1].expand(8, 64), W, o, C)]:
        with pytest.raises(ValueError):
            h.run_grouped(*args, "row", "bf16")
    with pytest.raises(ValueError):
        h.run_grouped_wgrad(A, A[:4], o, torch.zeros(3, 64, 64, device="cuda"), "bf16")


def test_repeated_calls_are_bit_identical(h):
    b = bounds_of([100, 31, 0, 500])
    A, W = draw((b[-1], 520), "bf16", 20), draw((4, 520, 384), "bf16", 21)
    first = run_forward(h, A, W, b, "row", "bf16")
    for _ in range(3):
        assert torch.equal(first, run_forward(h, A, W, b, "row", "bf16"))


def test_side_streams_and_graphs(h):
    """Work on a stream of the caller's choice, and captured in a CUDA graph
    whose replays follow the offsets' current values."""
    K, N = 128, 256
    A, W = draw((96, K), "bf16", 22), draw((3, K, N), "bf16", 23)
    A_d, W_d, o = A.cuda(), W.cuda(), device_offsets([0, 10, 60, 96])
    C = torch.zeros((96, N), device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    h.run_grouped(A_d, W_d, o, C, "row", "bf16", stream=side)
    h.sync_status(side)
    assert_close(C, *forward_ref(A, W, [0, 10, 60, 96]), K, "bf16")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h.run_grouped(A_d, W_d, o, C, "row", "bf16")
    for b in ([0, 96, 96, 96], [0, 0, 1, 96]):
        o.copy_(device_offsets(b))
        graph.replay()
        h.sync_status()
        assert_close(C, *forward_ref(A, W, b), K, "bf16")


def test_a_captured_workspace_outlives_growth(h):
    """Operands that are re-packed into the workspace: calls captured in a graph,
    then eager calls whose larger workspace replaces it, then the graph again."""
    b = bounds_of([30, 41])
    A, W = draw((71, 77), "bf16", 35), draw((2, 77, 131), "bf16", 36)
    A_d, W_d, o = A.cuda(), W.cuda(), device_offsets(b)
    C = torch.zeros((71, 131), device="cuda")
    h.run_grouped(A_d, W_d, o, C, "row", "bf16")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h.run_grouped(A_d, W_d, o, C, "row", "bf16")
    assert "+repackA+repackB" in h.last_path
    big = draw((3000, 1001), "bf16", 37), draw((4, 1001, 999), "bf16", 38)
    bb = bounds_of([1000, 0, 500, 1500])
    for _ in range(2):
        large = run_forward(h, *big, bb, "row", "bf16")
        C.zero_()
        graph.replay()
        h.sync_status()
        assert_close(C, *forward_ref(A, W, b), 77, "bf16")
        assert_close(large, *forward_ref(*big, bb), 1001, "bf16")


@pytest.mark.parametrize("tile", [1064, 2256, 41128])
@pytest.mark.parametrize("op", ["forward", "wgrad"])
def test_expired_wait_is_reported_and_the_handle_recovers(h, gm, op, tile):
    b = bounds_of([300, 200, 40])
    A, W, dC = draw((540, 256), "bf16", 24), draw((3, 256, 512), "bf16", 25), draw((540, 512), "bf16", 26)
    A_d, W_d, dC_d, o = A.cuda(), W.cuda(), dC.cuda(), device_offsets(b)
    C, g = torch.zeros((540, 512), device="cuda"), torch.zeros((3, 256, 512), device="cuda")
    h.set_option(gm.GEMM_OPT_GROUPED_TILE, tile)
    h.set_option(gm.GEMM_OPT_WAIT_TIMEOUT_NS, 20_000_000)

    def call():
        if op == "forward":
            h.run_grouped(A_d, W_d, o, C, "row", "bf16")
        else:
            h.run_grouped_wgrad(A_d, dC_d, o, g, "bf16")

    h.set_option(gm.GEMM_OPT_DEBUG_DROP_LOAD, 1)
    call()
    with pytest.raises(gm.GemmError) as e:
        h.sync_status()
    assert e.value.code == gm.GEMM_ERR_TIMEOUT
    h.set_option(gm.GEMM_OPT_DEBUG_DROP_LOAD, 0)
    call()
    h.sync_status()
    if op == "forward":
        assert_close(C, *forward_ref(A, W, b), 256, "bf16")
    else:
        assert_close(g, *wgrad_ref(A, dC, b), 300, "bf16")


def test_offsets_past_32_bits(h):
    """C of more than 2^32 elements: rows near the end land where they belong."""
    rows, K, N = 140_000, 64, 32_768
    A, W = draw((rows, K), "bf16", 27).cuda(), draw((2, K, N), "bf16", 28).cuda()
    C = torch.zeros((rows, N), dtype=torch.bfloat16, device="cuda")
    h.run_grouped(A, W, device_offsets([0, 131_000, rows]), C, "row", "bf16")
    h.sync_status()
    for r, g in ((0, 0), (65_600, 0), (130_999, 0), (131_000, 1), (rows - 1, 1)):
        row = torch.empty((1, N), device="cuda")
        h.run_grouped(A[r:r + 1], W[g:g + 1], device_offsets([0, 1]), row, "row", "bf16")
        a, w = A[r:r + 1].cpu().double(), W[g].cpu().double()
        assert_close(row, a @ w, a.abs() @ w.abs(), K, "bf16")
        assert torch.equal(C[r], row[0].bfloat16())
    assert int((C == 0).all(1).sum()) == 0


@pytest.mark.parametrize("layout", ["row", "col"])
@pytest.mark.parametrize("dtype", ["bf16", "tf32"])
def test_autograd_against_the_formula_and_differences(gm, dtype, layout):
    """The product is linear in each operand, so a central difference of any
    step is the directional derivative; small integers make both exact."""
    from dense_gemm_sm100_gb300.experts import grouped_matmul
    d = torch.bfloat16 if dtype == "bf16" else torch.float32
    gen = torch.Generator().manual_seed(29)
    b = bounds_of([40, 0, 70, 1], start=2)
    rows, K, N = b[-1] + 3, 72, 48

    def ints(*shape):
        return torch.randint(-2, 3, shape, generator=gen).to(d).cuda()

    A, W, dC = ints(rows, K), ints(4, K, N), ints(rows, N)
    B = W if layout == "row" else W.transpose(1, 2).contiguous()
    o = device_offsets(b)
    A.requires_grad_(), B.requires_grad_()
    C = grouped_matmul(A, B, o, layout, torch.float32)
    C.backward(dC.float())
    inside = torch.zeros(rows, dtype=torch.bool)
    inside[b[0]:b[-1]] = True
    assert (C[~inside.cuda()] == 0).all() and (A.grad[~inside.cuda()] == 0).all()
    dA_ref = forward_ref(dC.cpu(), W.cpu().transpose(1, 2), b)[0]
    dW_ref = wgrad_ref(A.detach().cpu(), dC.cpu(), b)[0]
    dB_ref = dW_ref if layout == "row" else dW_ref.transpose(1, 2)
    assert torch.equal(A.grad.cpu().double(), dA_ref.to(d).double())
    assert torch.equal(B.grad.cpu().double(), dB_ref.to(d).double())
    for which in (0, 1):
        V = ints(*(A if which == 0 else B).shape)

        def f(step):
            a = A.detach() + step * V if which == 0 else A.detach()
            w = B.detach() + step * V if which == 1 else B.detach()
            return (grouped_matmul(a, w, o, layout, torch.float32).double() * dC.double()).sum()

        diff = ((f(1) - f(-1)) / 2).item()
        ref = (V.cpu().double() * (dA_ref if which == 0 else dB_ref)).sum().item()
        assert diff == ref


def test_autograd_of_a_broadcast_output_gradient(gm):
    """sum() hands back an expanded gradient; a shared operand sums over its uses."""
    from dense_gemm_sm100_gb300.experts import grouped_matmul
    b = bounds_of([5, 12])
    gen = torch.Generator().manual_seed(30)
    A, W = (torch.randint(-2, 3, shape, generator=gen).float() for shape in ((17, 64), (2, 64, 128)))
    a, w = A.cuda().requires_grad_(), W.cuda().requires_grad_()
    o = device_offsets(b)
    (grouped_matmul(a, w, o).sum() + grouped_matmul(a, w, o).sum()).backward()
    ones = torch.ones(17, 128)
    assert torch.equal(a.grad.cpu().double(), 2 * forward_ref(ones, W.transpose(1, 2), b)[0])
    assert torch.equal(w.grad.cpu().double(), 2 * wgrad_ref(A, ones, b)[0])


def test_expert_layer_example(gm):
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_layer.py")
    spec = importlib.util.spec_from_file_location("expert_layer", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses, errors = example.main(["--tokens", "256", "--hidden", "256", "--inner", "320", "--experts", "8",
                                   "--steps", "4"])
    assert all(x > y for x, y in zip(losses, losses[1:]))
    # 4-bit rounding is off by 2^-2 of an element at most (1 and 1.5 of a step of 0.5), so the
    # two products of rounded operands stay well inside half of the output's norm
    assert all(e < 0.5 for e in errors.values())
