"""The router, the grouped products, the 8-bit experts and the orthogonalised update
together, as an expert layer uses them (examples/expert_layer.py)."""
import importlib.util
import os

import pytest
import torch
import torch.nn.functional as F

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_layer.py")
    spec = importlib.util.spec_from_file_location("expert_layer", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_runs_with_orthogonalised_updates(example):
    losses, errors = example.main(["--tokens", "130", "--hidden", "256", "--inner", "320", "--experts", "8", "--steps",
                                   "2", "--optimiser", "orthogonal"])
    assert len(losses) == 2 and all(v == v and v < float("inf") for v in losses)
    # 8-bit codes are off by half a step of 1/127 of a row's largest element, five times the
    # root mean square at most here: 5 / 254 = 2^-5.7 of an element's size for each of the
    # two operands of two products, four such errors in sequence
    assert all(e < 4 * 5 / 254 for (bits, _), e in errors.items() if bits == 8)


def test_gradients_of_the_layer(example):
    """Against the layer's formula in FP64 on the same choices.  Each gradient passes at
    most ten roundings to BF16, each off by at most 2^-8 of its tensor's norm: 10 * 2^-8."""
    torch.manual_seed(3)
    layer = example.ExpertLayer(192, 136, 7, 3)
    x = torch.randn(150, 192, device="cuda").bfloat16()
    g = torch.randn(150, 192, device="cuda").bfloat16().float()
    layer(x).float().backward(g)
    with torch.no_grad():
        chosen = example.route(x.float() @ layer.router.float().t(), 3)
    ref = {name: p.detach().double().requires_grad_() for name, p in layer.named_parameters()}
    score = torch.softmax(x.double() @ ref["router"].t(), -1).gather(1, chosen.expert)
    weight = score / score.sum(-1, keepdim=True)
    out = torch.zeros(150, 192, device="cuda", dtype=torch.float64)
    for choice in range(3):
        for e in range(7):
            at = (chosen.expert[:, choice] == e).nonzero().flatten()
            gate, up = (x[at].double() @ ref["gate_up"][e].t()).chunk(2, -1)
            y = (F.silu(gate) * up) @ ref["down"][e].t()
            out = out.index_add(0, at, y * weight[at, choice, None])
    out.backward(g.double())
    for name, p in layer.named_parameters():
        want = ref[name].grad
        assert (p.grad.double() - want).norm() <= 10 * 2 ** -8 * want.norm(), name


def test_updates_are_the_momentum_made_orthogonal(example):
    """Two steps by the optimiser against the same in FP64 on its BF16 momentum."""
    torch.manual_seed(4)
    w = torch.nn.Parameter(torch.zeros(3, 96, 64, device="cuda", dtype=torch.bfloat16))
    opt = example.ExpertUpdates([w], lr=1.0)
    for step in range(2):
        w.grad = torch.randn_like(w)
        before = w.detach().double()
        opt.step()
        X = opt.state[w]["momentum"].double()
        X = X / X.norm(dim=(-2, -1), keepdim=True)
        for _ in range(5):
            A = X @ X.mT
            X = 3.4445 * X + (-4.7750 * A + 2.0315 * A @ A) @ X
        want = before - X * 1.5 ** 0.5
        # the update's and the sum's roundings, 2^-8 each, and the kernel's own within one more
        assert (w.detach().double() - want).norm() <= 3 * 2 ** -8 * want.norm()


@pytest.mark.parametrize("tokens,experts,k", [(40, 12, 3), (1, 5, 2), (300, 64, 4), (700, 8, 2)])
def test_captured_serving_with_padding(tokens, experts, k):
    """Router, quantisation and grouped 8-bit product as one captured graph, replayed on
    other tokens: some, none and all of them padding (logits of minus infinity), whose rows
    stay as they are.  Exact integer sums: the result is the formula's, rounded."""
    from dense_gemm_sm100_gb300 import gemm
    K, N = 80, 50
    gen = torch.Generator().manual_seed(5)
    router = torch.randn((K, experts), generator=gen).cuda()
    x, pad = torch.zeros((tokens, K), device="cuda"), torch.zeros(tokens, dtype=torch.bool, device="cuda")
    with gemm.Gemm(0) as h:
        w = h.i8_quantise(torch.randn((experts, N, K), generator=gen).cuda(), gemm.i8_empty(experts * N, K))
        r, xq = gemm.routing_empty(tokens, experts, k), gemm.i8_empty(tokens * k, K)
        y = torch.empty((tokens * k, N), device="cuda")

        def serve():
            logits = (x @ router).masked_fill(pad[:, None], float("-inf"))
            h.route(logits, r)
            h.i8_quantise(x[r.order // k], xq)
            y.fill_(7.0)
            h.run_i8_grouped(xq, w, r.offsets, y)

        serve()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            serve()
        for share in (0.0, 0.4, 1.0):
            x.copy_(torch.randn((tokens, K), generator=gen))
            pad.copy_(torch.rand(tokens, generator=gen) < share)
            graph.replay()
            h.sync_status()
            bounds = r.offsets.tolist()
            assert bounds[0] == int(pad.sum()) * k and bounds[-1] == tokens * k
            assert (y[:bounds[0]] == 7).all() and (r.expert[pad] == -1).all() and (r.weights[pad] == 0).all()
            codes, wide = xq.codes[:, :K].double(), w.codes[:, :K].double()
            for e in range(experts):
                rows, cols = slice(bounds[e], bounds[e + 1]), slice(e * N, (e + 1) * N)
                assert (r.expert.flatten()[r.order[rows]] == e).all()
                sums = codes[rows] @ wide[cols].t()
                want = (sums.float() * xq.scales[rows, None]) * w.scales[cols]
                assert torch.equal(y[rows], want)


def test_two_threads_with_a_handle_each():
    """Calls of all three at the same time, on a stream and a handle a thread."""
    import threading
    from dense_gemm_sm100_gb300 import gemm
    gen = torch.Generator().manual_seed(6)
    logits, G = torch.randn((500, 24), generator=gen).cuda(), torch.randn((2, 90, 130), generator=gen).cuda()
    A, B = torch.randn((60, 200), generator=gen).cuda(), torch.randn((70, 200), generator=gen).cuda()

    def work(h):
        r = h.route(logits, gemm.routing_empty(500, 24, 3))
        a, b = h.i8_quantise(A, gemm.i8_empty(60, 200)), h.i8_quantise(B, gemm.i8_empty(70, 200))
        return [*r, h.run_i8(a, b, torch.empty((60, 70), device="cuda")), h.orthogonalise(G, torch.empty_like(G))]

    with gemm.Gemm(0) as h:
        want = work(h)
        torch.cuda.synchronize()
    got, wrong = [None] * 4, []

    def loop(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()), gemm.Gemm(0) as h:
                for _ in range(20):
                    got[i] = work(h)
                h.sync_status()
        except Exception as e:  # noqa: BLE001 - reported by the assertion below
            wrong.append(e)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=loop, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong
    torch.cuda.synchronize()
    for result in got:
        for a, b in zip(result, want):
            assert torch.equal(a, b)
