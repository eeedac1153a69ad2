"""The handle's workspace on the GPU: captured calls and calls on several
streams.  Operands have odd pitches, so every call re-packs them into the
workspace.  Small integers make all sums exact (at most 4 * 77 in FP32), so
results are compared bit for bit."""
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


class Call:
    """A grouped product of two experts, or a dense product, at odd sizes."""

    def __init__(self, grouped, rows, K, N, seed):
        gen = torch.Generator().manual_seed(seed)
        ints = lambda *s: torch.randint(-2, 3, s, generator=gen).bfloat16().cuda()
        self.A, self.B = ints(rows, K), ints(*((2, K, N) if grouped else (K, N)))
        self.C = torch.zeros((rows, N), device="cuda")
        self.offsets = torch.tensor([0, rows // 3, rows], device="cuda") if grouped else None
        a, b, cut = self.A.float(), self.B.float(), rows // 3
        self.ref = torch.cat([a[:cut] @ b[0], a[cut:] @ b[1]]) if grouped else a @ b
        torch.cuda.synchronize()

    def run(self, h, stream=None):
        if self.offsets is not None:
            h.run_grouped(self.A, self.B, self.offsets, self.C, "row", "bf16", stream=stream)
        else:
            h.run(self.A, self.B, self.C, "row", "bf16", stream=stream)
        assert "+repackA+repackB" in h.last_path

    def right(self):
        ok = torch.equal(self.C, self.ref)
        self.C.zero_()
        return ok


@pytest.mark.parametrize("grouped", [False, True], ids=["dense", "grouped"])
def test_the_first_call_of_a_handle_is_captured(h, grouped):
    call, other, large = Call(grouped, 71, 77, 131, 1), Call(grouped, 60, 75, 130, 2), Call(grouped, 3001, 77, 999, 3)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call.run(h)
    other.run(h)  # fits into the workspace, and the graph has not run yet
    h.sync_status()
    assert other.right()
    for _ in range(3):
        graph.replay()
        h.sync_status()
        assert call.right()
        large.run(h)  # outgrows it the first time
        h.sync_status()
        assert large.right()


@pytest.mark.parametrize("grouped", [False, True], ids=["dense", "grouped"])
def test_the_workspace_grows_while_a_call_is_captured(h, grouped):
    small, large = Call(grouped, 60, 75, 130, 4), Call(grouped, 3001, 77, 999, 5)
    small.run(h)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        large.run(h)
    for _ in range(2):
        small.run(h)
        graph.replay()
        small.run(h)
        h.sync_status()
        assert small.right() and large.right()


@pytest.mark.parametrize("grouped", [False, True], ids=["dense", "grouped"])
def test_calls_on_streams_that_nothing_orders(h, grouped):
    calls = [Call(grouped, 1501 + 100 * i, 77, 999, 10 + i) for i in range(4)]
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(5):
        for i in range(12):
            calls[i % 4].run(h, streams[i % 3])
        for s in streams:
            h.sync_status(s)
        assert all(c.right() for c in calls)
        torch.cuda.synchronize()
