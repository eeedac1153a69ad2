"""``experts.grouped_matmul`` on the GPU beyond its first gradients."""
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


def offsets_of(sizes, start=0):
    b = [start]
    for s in sizes:
        b.append(b[-1] + s)
    return torch.tensor(b, dtype=torch.int64, device="cuda")


@pytest.mark.parametrize("layout", ["row", "col"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_second_order_gradients_are_the_formulas(gm, dtype, layout):
    """With gA = dC B^T and gB = A^T dC, the gradient of sum(gA U) + sum(gB V) is
    dC V^T in A, U^T dC in B and U B + A V in dC.  Small integers make every
    sum exact (at most 4 * 72 * 4 in FP32), so each is its value in 64 bits
    rounded once to the operand's type."""
    from dense_gemm_sm100_gb300.experts import grouped_matmul
    gen = torch.Generator().manual_seed(51)
    sizes, K, N = [40, 0, 70, 1], 72, 48
    rows = sum(sizes) + 5

    def ints(*shape):
        return torch.randint(-2, 3, shape, generator=gen).to(dtype).cuda()

    A, W, dC, U, V = ints(rows, K), ints(4, K, N), ints(rows, N), ints(rows, K), ints(4, K, N)
    lay = (lambda t: t) if layout == "row" else (lambda t: t.transpose(1, 2).contiguous())
    o = offsets_of(sizes, 2)
    a, w, d = A.clone().requires_grad_(), lay(W).requires_grad_(), dC.clone().requires_grad_()
    gA, gB = torch.autograd.grad(grouped_matmul(a, w, o, layout), (a, w), d, create_graph=True)
    got = torch.autograd.grad((gA * U).sum() + (gB * lay(V)).sum(), (a, w, d))
    b = o.tolist()
    A, W, dC, U, V = (t.detach().double() for t in (A, W, dC, U, V))
    dA = torch.zeros(rows, K, dtype=torch.float64, device="cuda")
    first, second = (torch.zeros(rows, N, dtype=torch.float64, device="cuda") for _ in range(2))
    dW = torch.zeros_like(W)
    for g in range(4):
        s = slice(b[g], b[g + 1])
        dA[s] = dC[s] @ V[g].T
        dW[g] = U[s].T @ dC[s]
        first[s], second[s] = U[s] @ W[g], A[s] @ V[g]
    assert torch.equal(got[0], dA.to(dtype))
    assert torch.equal(got[1], lay(dW).to(dtype))
    assert torch.equal(got[2], first.to(dtype) + second.to(dtype))


@pytest.mark.parametrize("layout", ["row", "col"])
@pytest.mark.parametrize("bad", [[0, 5, 3, 8], [0, 2, 3, 9]])
def test_refused_offsets_give_defined_results_and_are_reported(gm, bad, layout):
    from dense_gemm_sm100_gb300.experts import grouped_matmul
    a = torch.ones((8, 64), device="cuda").bfloat16().requires_grad_()
    w = torch.ones((3, 64, 64), device="cuda").bfloat16().requires_grad_()
    with gm.Gemm(0) as h:
        y = grouped_matmul(a, w, torch.tensor(bad, device="cuda"), layout, handle=h)
        y.sum().backward()
        assert (y == 0).all() and (a.grad == 0).all() and torch.isnan(w.grad).all()
        with pytest.raises(gm.GemmError) as e:
            h.sync_status()
        assert e.value.code == gm.GEMM_ERR_INVALID
        a.grad = w.grad = None
        y = grouped_matmul(a, w, torch.tensor([0, 2, 3, 8], device="cuda"), layout, handle=h)
        y.sum().backward()
        h.sync_status()
        assert (y == 64).all() and (a.grad == 64).all()
        assert (w.grad == torch.tensor([2, 1, 5], device="cuda").view(3, 1, 1)).all()


def test_streams_and_threads_share_the_default_handle(gm):
    """Operands with odd pitches go through the handle's workspace; small
    integers make forward and backward exact (sums of at most 4 * 300 in FP32
    before the rounding to the operand's type)."""
    import threading
    from dense_gemm_sm100_gb300.experts import grouped_matmul
    sizes, K, N = [300, 0, 211], 77, 131
    o = offsets_of(sizes)

    def work(seed, results):
        gen = torch.Generator().manual_seed(seed)
        ints = lambda *s: torch.randint(-2, 3, s, generator=gen).bfloat16().cuda()
        stream = torch.cuda.Stream()
        ok = True
        for _ in range(6):
            A, W, dC = ints(sum(sizes), K), ints(3, K, N), ints(sum(sizes), N)
            stream.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(stream):
                a, w = A.clone().requires_grad_(), W.clone().requires_grad_()
                y = grouped_matmul(a, w, o, "row", torch.float32)
                y.backward(dC.float())
                stream.synchronize()
            ref = torch.cat([A[:300].float() @ W[0].float(), A[300:].float() @ W[2].float()])
            dA = torch.cat([dC[:300].float() @ W[0].float().T, dC[300:].float() @ W[2].float().T])
            dW = torch.stack([A[:300].float().T @ dC[:300].float(), torch.zeros(K, N, device="cuda"),
                              A[300:].float().T @ dC[300:].float()])
            ok = ok and torch.equal(y, ref) and torch.equal(a.grad, dA.bfloat16()) and torch.equal(w.grad, dW.bfloat16())
        results.append(ok)

    results = []
    threads = [threading.Thread(target=work, args=(60 + i, results)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    gm.default_handle().sync_status()
    assert results == [True] * 3
