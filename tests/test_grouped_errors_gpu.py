"""What C holds after a grouped call that went wrong on the GPU, with the flag
that turns unwritten elements into NaN.

Waits are made to run out by dropping one stage's loads (the library's test
hook); the handle reports it and stays usable.  Bounds of the elements that
were computed: (K + 2) 2^-23 S, S = sum |a b| over K terms."""
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


def draw(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()


@pytest.mark.parametrize("tile", [0, 1128, 1256, 2128, 2256, 41128])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bad", [[0, 5, 3, 600], [-1, 2, 3, 600], [0, 2, 3, 601]])
def test_refused_weight_gradients(h, gm, bad, out, tile):
    h.set_option(gm.GEMM_OPT_GROUPED_TILE, tile)
    h.set_option(gm.GEMM_OPT_MAX_CTAS, 4)
    A, B = draw((600, 200), 1), draw((600, 333), 2)
    store = torch.full((3, 203, 340), 7.0, dtype=out, device="cuda")
    C = store[:, 1:201, 3:336]
    o = torch.tensor(bad, device="cuda")
    for nan in (False, True):
        h.run_grouped_wgrad(A, B, o, C, "bf16", nan_on_error=nan)
        with pytest.raises(gm.GemmError) as e:
            h.sync_status()
        assert e.value.code == gm.GEMM_ERR_INVALID
        assert torch.isnan(C).all() if nan else (C == 7).all()
        rest = store.clone()
        rest[:, 1:201, 3:336] = 7
        assert (rest == 7).all()
    rows = torch.full((600, 333), 7.0, dtype=out, device="cuda")
    h.run_grouped(A, draw((3, 200, 333), 3), o, rows, "row", "bf16", nan_on_error=True)
    with pytest.raises(gm.GemmError):
        h.sync_status()
    assert (rows == 7).all()  # no rows are the call's own


@pytest.mark.parametrize("ctas", [0, 4], ids=["all", "few"])
@pytest.mark.parametrize("tile", [1064, 1128, 2128, 2256, 21128, 41064])
@pytest.mark.parametrize("K", [256, 1700])
@pytest.mark.parametrize("op", ["forward", "wgrad"])
def test_expired_waits(h, gm, op, K, tile, ctas):
    """K = 1700: sums in segments."""
    h.set_option(gm.GEMM_OPT_GROUPED_TILE, tile)
    h.set_option(gm.GEMM_OPT_MAX_CTAS, ctas)
    h.set_option(gm.GEMM_OPT_WAIT_TIMEOUT_NS, 20_000_000)
    N = 520
    if op == "forward":
        b = [3, 303, 303, 503, 543]
        A, B = draw((550, K), 4), draw((4, K, N), 5)
        C = torch.full((550, N + 4), 7.0, device="cuda")
        ref, S = torch.full((550, N), 7.0, dtype=torch.float64, device="cuda"), torch.zeros(550, N, device="cuda").double()
        for g in range(4):
            s = slice(b[g], b[g + 1])
            ref[s], S[s] = A[s].double() @ B[g].double(), A[s].double().abs() @ B[g].double().abs()
        own = torch.zeros_like(ref, dtype=torch.bool)
        own[b[0]:b[-1]] = True
        call = lambda: h.run_grouped(A, B, o, C[:, :N], "row", "bf16", nan_on_error=True)
    else:
        b = [3, 3 + K, 3 + K, K + 43, K + 50]
        A, B = draw((K + 60, 300), 6), draw((K + 60, N), 7)
        C = torch.full((4, 300, N + 4), 7.0, device="cuda")
        ref, S = (torch.stack([f(A[b[g]:b[g + 1]].double()).T @ f(B[b[g]:b[g + 1]].double()) for g in range(4)])
                  for f in (lambda t: t, torch.abs))
        own = torch.ones_like(ref, dtype=torch.bool)
        call = lambda: h.run_grouped_wgrad(A, B, o, C[:, :, :N], "bf16", nan_on_error=True)
    o = torch.tensor(b, device="cuda")

    def right():
        return (C[..., :N].double() - ref).abs() <= (K + 2) * 2.0 ** -23 * S

    h.set_option(gm.GEMM_OPT_DEBUG_DROP_LOAD, 1)
    call()
    with pytest.raises(gm.GemmError) as e:
        h.sync_status()
    assert e.value.code == gm.GEMM_ERR_TIMEOUT
    nan = torch.isnan(C[..., :N])
    assert nan.any() and not (nan & ~own).any() and (right() | nan).all() and (C[..., N:] == 7).all()
    h.set_option(gm.GEMM_OPT_DEBUG_DROP_LOAD, 0)
    call()
    h.sync_status()
    assert right().all() and (C[..., N:] == 7).all()
