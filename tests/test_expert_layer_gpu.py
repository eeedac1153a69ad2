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
