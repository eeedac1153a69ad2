"""The router's weights as torch operations (the gradients of gradients): rows
without choices add nothing, whatever their logits hold."""
import math

import pytest
import torch

from dense_gemm_sm100_gb300.experts import _weights_of


@pytest.mark.parametrize("renormalise", [True, False])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_rows_without_choices_have_zero_gradients(scoring, renormalise, bad):
    x = torch.randn((4, 6), generator=torch.Generator().manual_seed(1))
    expert = torch.tensor([[2, 0], [-1, -1], [5, -1], [-1, -1]])
    x[1, 0] = bad  # a row that holds one: its index 0 stands in for the choices that are not there
    x[3] = bad
    leaf = x.clone().requires_grad_()
    w = _weights_of(leaf, expert, scoring, renormalise, 1.5)
    assert (w[[1, 3]] == 0).all() and w[2, 1] == 0
    dw = torch.tensor([[1.0, -2.0], [3.0, 4.0], [0.5, 7.0], [1.0, 1.0]])
    first, = torch.autograd.grad(w, leaf, dw, create_graph=True)
    second, = torch.autograd.grad(first.square().sum(), leaf)
    for g in (first, second):
        assert torch.isfinite(g).all()
        assert (g[[1, 3]] == 0).all()
    # the other rows as if they stood alone
    alone = x[[0, 2]].clone().requires_grad_()
    a, = torch.autograd.grad(_weights_of(alone, expert[[0, 2]], scoring, renormalise, 1.5), alone, dw[[0, 2]],
                             create_graph=True)
    b, = torch.autograd.grad(a.square().sum(), alone)
    assert torch.equal(first[[0, 2]], a) and torch.equal(second[[0, 2]], b)


@pytest.mark.parametrize("renormalise", [True, False])
def test_choices_far_below_the_other_slots(renormalise):
    """Two equal choices share the weight however low their logits are, with a slot that
    holds no choice beside them."""
    x = torch.full((3, 4), -math.inf)
    x[:, 1:3] = torch.tensor([[-1e31], [-3e38], [5.0]])
    expert = torch.tensor([[1, 2, -1]] * 3)
    leaf = x.clone().requires_grad_()
    w = _weights_of(leaf, expert, "softmax", renormalise, 1.0)
    assert torch.equal(w, torch.tensor([[0.5, 0.5, 0.0]] * 3))
    first, = torch.autograd.grad(w, leaf, torch.tensor([[1.0, -1.0, 9.0]] * 3), create_graph=True)
    second, = torch.autograd.grad(first.square().sum(), leaf)
    assert torch.equal(first.detach(), torch.tensor([[0.0, 0.5, -0.5, 0.0]] * 3))
    assert torch.isfinite(second).all()
