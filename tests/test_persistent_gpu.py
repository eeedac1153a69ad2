"""Grouped products whose CTAs run many tiles one after another, on the GPU:
four CTAs (two pairs) share each launch, so rings wrap across tiles, both
accumulators are handed back and forth between tiles, and long sums leave an
odd or an even number of segments behind each tile.

Bounds as for the other grouped products, S = sum |a b| over K terms:
(K + 2) 2^-23 S; TF32 operands add 2^-9 + 2^-20 of S; BF16 results round by
2^-8 of themselves on top."""
import pytest
import torch

pytestmark = pytest.mark.gpu

TILES = [1032, 1064, 1128, 1224, 1256, 2032, 2064, 2128, 2224, 2256]


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
        handle.set_option(gm.GEMM_OPT_MAX_CTAS, 4)
        yield handle


def draw(shape, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=gen).to(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()


def edges(sizes):
    b = [0]
    for s in sizes:
        b.append(b[-1] + s)
    return b


def assert_close(C, ref, S, K, dtype):
    t = (K + 2) * 2.0 ** -23 * S
    if dtype == "tf32":
        t = t + (2.0 ** -9 + 2.0 ** -20) * S
    if C.dtype == torch.bfloat16:
        t = t + 2.0 ** -8 * (ref.abs() + t)
    over = ~((C.double() - ref).abs() <= t)
    assert not over.any(), f"{int(over.sum())} elements off"


# ring stages of 64 (BF16) and 32 (TF32) elements; segments of 12 and 8 stages
@pytest.mark.parametrize("dtype,K", [("bf16", 264), ("bf16", 1500), ("bf16", 2100), ("tf32", 136), ("tf32", 500),
                                     ("tf32", 700)])
@pytest.mark.parametrize("layout", ["row", "col"])
@pytest.mark.parametrize("tile", TILES)
def test_forward(h, gm, tile, layout, dtype, K):
    h.set_option(gm.GEMM_OPT_GROUPED_TILE, tile)
    sizes, N = [300, 0, 17, 128, 257, 1], 392
    b = edges(sizes)
    A, W = draw((b[-1], K), dtype, 1), draw((6, K, N), dtype, 2)
    B = W if layout == "row" else W.transpose(1, 2).contiguous()
    o = torch.tensor(b, device="cuda")
    ref, S = (torch.cat([f(A[b[g]:b[g + 1]].double()) @ f(W[g].double()) for g in range(6)])
              for f in (lambda t: t, torch.abs))
    for out in (torch.float32, torch.bfloat16) if dtype == "bf16" else (torch.float32,):
        C = torch.full((b[-1], N), float("nan"), dtype=out, device="cuda")
        h.run_grouped(A, B, o, C, layout, dtype)
        h.sync_status()
        assert_close(C, ref, S, K, dtype)


@pytest.mark.parametrize("tile", [1128, 1256, 2128, 2256])
@pytest.mark.parametrize("dtype,sizes", [("bf16", [1500, 0, 17, 2100, 64, 700]), ("tf32", [500, 0, 17, 700, 64, 200]),
                                         ("bf16", [300, 0, 17, 64, 1, 131]), ("tf32", [30, 0, 17, 64, 1, 70])])
@pytest.mark.parametrize("MN", [(300, 392), (512, 256), (257, 1031)])
def test_wgrad(h, gm, MN, dtype, sizes, tile):
    """Groups of no, one, two and three segments side by side, and launches
    short enough not to be cut."""
    h.set_option(gm.GEMM_OPT_GROUPED_TILE, tile)
    M, N = MN
    b = edges(sizes)
    A, B = draw((b[-1], M), dtype, 3), draw((b[-1], N), dtype, 4)
    o = torch.tensor(b, device="cuda")
    ref, S = (torch.stack([f(A[b[g]:b[g + 1]].double()).T @ f(B[b[g]:b[g + 1]].double()) for g in range(6)])
              for f in (lambda t: t, torch.abs))
    for out in (torch.float32, torch.bfloat16) if dtype == "bf16" else (torch.float32,):
        C = torch.full((6, M, N), float("nan"), dtype=out, device="cuda")
        h.run_grouped_wgrad(A, B, o, C, dtype)
        h.sync_status()
        assert_close(C, ref, S, max(sizes), dtype)
        assert (C[1] == 0).all()
