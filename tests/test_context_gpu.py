"""Calls from a thread whose current CUDA context is one of its own making, beside
the primary one that torch and a handle made there use."""
import ctypes

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


class Driver:
    def __init__(self):
        self.lib = ctypes.CDLL("libcuda.so.1")

    def __getattr__(self, name):
        f = getattr(self.lib, name)

        def call(*args):
            rc = f(*args)
            assert rc == 0, (name, rc)

        return call

    def current(self):
        c = ctypes.c_void_p()
        self.cuCtxGetCurrent(ctypes.byref(c))
        return c.value


@pytest.fixture()
def own(gm):
    """A context of this test's own, current while it runs."""
    torch.zeros(1, device="cuda")
    d = Driver()
    primary = d.current()
    ctx = ctypes.c_void_p()
    d.cuCtxCreate_v2(ctypes.byref(ctx), 0, 0)
    assert d.current() == ctx.value != primary
    d.context, d.primary = ctx.value, primary
    yield d
    assert d.current() == ctx.value
    d.cuCtxPopCurrent_v2(ctypes.byref(ctypes.c_void_p()))
    d.cuCtxDestroy_v2(ctx)
    assert d.current() == primary


def test_calls_on_a_handle_of_the_primary_context(gm, own):
    """They work in the primary context and leave the thread's own one current."""
    d = own
    d.cuCtxPushCurrent_v2(ctypes.c_void_p(d.primary))
    A = torch.ones((96, 64), device="cuda").bfloat16()
    B = torch.ones((2, 64, 64), device="cuda").bfloat16()
    offsets = torch.tensor([0, 40, 96], device="cuda")
    C, D, O = (torch.zeros(s, device="cuda") for s in ((96, 64), (96, 64), (64, 64)))
    r = gm.routing_empty(96, 8, 2)
    x = torch.randn((96, 8), device="cuda")
    q, w, Y = gm.i8_empty(96, 64), gm.i8_empty(128, 64), torch.zeros((96, 64), device="cuda")
    handle = gm.Gemm(0)
    torch.cuda.synchronize()
    d.cuCtxPopCurrent_v2(ctypes.byref(ctypes.c_void_p()))
    assert d.current() == d.context
    for call in (lambda: handle.run(A, B[0], D, "row", "bf16", stream=0),
                 lambda: handle.run_grouped(A, B, offsets, C, stream=0),
                 lambda: handle.i8_quantise(A, q, stream=0),
                 lambda: handle.i8_quantise(B.view(128, 64), w, stream=0),
                 lambda: handle.run_i8_grouped(q, w, offsets, Y, stream=0),
                 lambda: handle.route(x, r, stream=0),
                 lambda: handle.orthogonalise(D[:64], O, stream=0),
                 lambda: handle.sync_status(stream=0)):
        call()
        assert d.current() == d.context
    d.cuCtxPushCurrent_v2(ctypes.c_void_p(d.primary))
    assert (C == 64).all() and (D == 64).all() and torch.allclose(Y, C, rtol=1e-6)
    assert (torch.sort(x, 1, descending=True).indices[:, :2] == r.expert).all()
    assert torch.isfinite(O).all()
    handle.close()
    d.cuCtxPopCurrent_v2(ctypes.byref(ctypes.c_void_p()))


def test_a_handle_made_in_the_threads_own_context(gm, own):
    """Its memory, kernels and calls belong to that context, which stays current; the
    kernels' use in the primary one before does not count for it."""
    d = own
    M, N, K = 4, 64, 16384  # 64 KB of shared memory, which a kernel has to be allowed
    d.cuCtxPushCurrent_v2(ctypes.c_void_p(d.primary))
    q, w, C = gm.i8_empty(M, K), gm.i8_empty(N, K), torch.zeros((M, N), device="cuda")
    for t in (q, w):
        t.codes.fill_(1)
        t.scales.fill_(1.0)
    with gm.Gemm(0) as there:
        there.run_i8(q, w, C)
        there.sync_status()
    assert (C == K).all()
    d.cuCtxPopCurrent_v2(ctypes.byref(ctypes.c_void_p()))
    handle = gm.Gemm(0)
    assert d.current() == d.context
    codes, scales = bytes(range(1, 65)) * (K // 64), (ctypes.c_float * 64)(*[1.0] * 64)
    want = float(sum(v * v for v in codes))

    def memory(size, source=None):
        p = ctypes.c_uint64()
        d.cuMemAlloc_v2(ctypes.byref(p), ctypes.c_size_t(size))
        if source is not None:
            d.cuMemcpyHtoD_v2(p, source, ctypes.c_size_t(size))
        return p

    a, b = memory(M * K, codes * M), memory(N * K, codes * N)
    s, c = memory(4 * 64, scales), memory(4 * M * N)
    rc = gm.gemm_i8_run(handle.handle, M, N, K, a.value, K, s.value, b.value, K, s.value, c.value, N, gm.GEMM_F32, 0)
    assert rc == 0 and d.current() == d.context
    handle.sync_status(stream=0)
    got = (ctypes.c_float * (M * N))()
    d.cuMemcpyDtoH_v2(got, c, ctypes.c_size_t(4 * M * N))
    assert all(v == want for v in got)
    handle.close()
    assert d.current() == d.context
    for p in (a, b, s, c):
        d.cuMemFree_v2(p)
