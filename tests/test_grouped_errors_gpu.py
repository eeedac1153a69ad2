"""Weight gradients that went wrong on the GPU, with the flag that makes them
NaN.  A wait is made to run out by dropping one stage's loads (the library's
test hook); the handle reports it and stays usable."""
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


def ints(shape, seed):
    return torch.randint(-2, 3, shape, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,bad", [(600, [0, 5, 3, 600]), (600, [-1, 2, 3, 600]), (600, [0, 2, 3, 601]),
                                      (600, [0, 9, 5, 2]), (0, [0, 0, 0, 1])])
def test_refused_offsets(h, gm, rows, bad, out):
    A, B = ints((rows, 200), 1), ints((rows, 333), 2)
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


@pytest.mark.parametrize("tile", [0, 1128, 2256, 21128])
def test_expired_wait(h, gm, tile):
    """NaN until the handle has reported it; sums of small integers are exact."""
    h.set_option(gm.GEMM_OPT_GROUPED_TILE, tile)
    h.set_option(gm.GEMM_OPT_WAIT_TIMEOUT_NS, 20_000_000)
    A, B, b = ints((600, 200), 3), ints((600, 333), 4), [3, 303, 303, 590]
    ref = torch.stack([A[b[g]:b[g + 1]].float().T @ B[b[g]:b[g + 1]].float() for g in range(3)])
    o = torch.tensor(b, device="cuda")
    C = torch.full((3, 200, 333), 7.0, device="cuda")

    def run():
        h.run_grouped_wgrad(A, B, o, C, "bf16", nan_on_error=True)

    h.set_option(gm.GEMM_OPT_DEBUG_DROP_LOAD, 1)
    run()
    h.set_option(gm.GEMM_OPT_DEBUG_DROP_LOAD, 0)
    torch.cuda.synchronize()
    assert torch.isnan(C).all()
    run()
    torch.cuda.synchronize()
    assert torch.isnan(C).all()
    with pytest.raises(gm.GemmError) as e:
        h.sync_status()
    assert e.value.code == gm.GEMM_ERR_TIMEOUT
    run()
    h.sync_status()
    assert torch.equal(C, ref)


def test_many_groups(h, gm):
    """More groups than a block has threads, the last pair of offsets wrong."""
    G = 4096
    A, B = ints((G, 8), 5), ints((G, 8), 6)
    o = torch.arange(G + 1, device="cuda")
    C = torch.full((G, 8, 8), 7.0, device="cuda")
    h.run_grouped_wgrad(A, B, o, C, "bf16", nan_on_error=True)
    h.sync_status()
    assert torch.equal(C, A.float()[:, :, None] * B.float()[:, None, :])
    o[G] = G + 1
    h.run_grouped_wgrad(A, B, o, C, "bf16", nan_on_error=True)
    with pytest.raises(gm.GemmError):
        h.sync_status()
    assert torch.isnan(C).all()
