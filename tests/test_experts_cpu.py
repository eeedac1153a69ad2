"""The autograd functions around the grouped products, without a GPU: a
stand-in handle computes what the library computes, in the same places."""
import pytest
import torch

from dense_gemm_sm100_gb300 import experts, gemm as g


class StandIn:
    """``Gemm``'s two grouped calls in torch, with their contract: rows outside
    the groups are not touched, a group without rows gets a zero weight
    gradient, and nothing is known to autograd."""

    refuse = False  # as the kernels do with offsets that decrease: compute nothing

    @torch.no_grad()
    def run_grouped(self, A, B, offsets, C, layout, dtype):
        b = offsets.tolist()
        for i in range(B.shape[0]):
            W = B[i] if layout == g.GEMM_B_ROW_MAJOR else B[i].t()
            if not self.refuse:
                C[b[i]:b[i + 1]] = (A[b[i]:b[i + 1]] @ W).to(C.dtype)
        return C

    @torch.no_grad()
    def run_grouped_wgrad(self, A, B, offsets, C, dtype, nan_on_error=False):
        b = offsets.tolist()
        if self.refuse and nan_on_error:
            C.fill_(float("nan"))
        for i in range(C.shape[0]):
            if not self.refuse:
                C[i] = (A[b[i]:b[i + 1]].t() @ B[b[i]:b[i + 1]]).to(C.dtype)
        return C


def product(A, B, offsets, layout, handle=None):
    return experts._product(A, B, offsets, layout, g.GEMM_TF32, A.dtype, handle or StandIn())


def formula(A, B, b, layout):
    """The product from torch operations, zeros for rows of no group."""
    out = [A.new_zeros(b[0], B.shape[2 if layout == g.GEMM_B_ROW_MAJOR else 1])]
    for i in range(B.shape[0]):
        out.append(A[b[i]:b[i + 1]] @ (B[i] if layout == g.GEMM_B_ROW_MAJOR else B[i].t()))
    return torch.cat(out + [out[0].new_zeros(A.shape[0] - b[-1], out[0].shape[1])])


def operands(layout, seed=0):
    gen = torch.Generator().manual_seed(seed)
    b = [1, 4, 4, 9]  # an empty group, and a row outside the groups at either end
    K, N = 3, 2
    A = torch.randn((10, K), generator=gen, dtype=torch.float64)
    B = torch.randn((3, K, N) if layout == g.GEMM_B_ROW_MAJOR else (3, N, K), generator=gen, dtype=torch.float64)
    return A.requires_grad_(), B.requires_grad_(), b


LAYOUTS = [g.GEMM_B_ROW_MAJOR, g.GEMM_B_COL_MAJOR]


@pytest.mark.parametrize("layout", LAYOUTS)
def test_gradients_against_differences(layout):
    A, B, b = operands(layout)
    f = lambda x, w: product(x, w, torch.tensor(b), layout)
    assert torch.autograd.gradcheck(f, (A, B))
    assert torch.autograd.gradgradcheck(f, (A, B))


@pytest.mark.parametrize("layout", LAYOUTS)
def test_a_gradient_penalty_has_the_formulas_gradient(layout):
    """Gradients of sum(y^2) + sum(gA^2) + sum(gB^2): linear sums of products,
    the same in both forms up to rounding (64 bits, terms of order 100)."""
    got = []
    for f in (lambda x, w, b: product(x, w, torch.tensor(b), layout), lambda x, w, b: formula(x, w, b, layout)):
        A, B, b = operands(layout, 1)
        y = f(A, B, b)
        gA, gB = torch.autograd.grad(y.pow(2).sum(), (A, B), create_graph=True)
        assert gA.requires_grad and gB.requires_grad
        got.append(torch.autograd.grad(y.pow(2).sum() + gA.pow(2).sum() + gB.pow(2).sum(), (A, B)))
    for x, ref in zip(*got):
        torch.testing.assert_close(x, ref, rtol=1e-10, atol=1e-10)


def test_a_gradient_penalty_of_operands_that_are_copied():
    """A transposed view and an expanded one: the copies that the kernels read
    are part of the graph."""
    got = []
    for f in (lambda x, w, b: product(x, w, torch.tensor(b), 0), lambda x, w, b: formula(x, w, b, 0)):
        A, B, b = operands(0, 2)
        view, wide = A.detach().t().clone().requires_grad_(), B.detach()[:1].clone().requires_grad_()
        y = f(view.t(), wide.expand(3, -1, -1), b)
        grads = torch.autograd.grad(y.sin().sum(), (view, wide), create_graph=True)
        got.append(torch.autograd.grad(sum(x.pow(2).sum() for x in grads), (view, wide)))
    for x, ref in zip(*got):
        torch.testing.assert_close(x, ref, rtol=1e-10, atol=1e-10)


@pytest.mark.parametrize("layout", LAYOUTS)
def test_a_refused_call_leaves_no_unwritten_memory(layout):
    """Where the kernels compute nothing, the output and dA are zero and dB is
    NaN everywhere, whatever the allocator hands out."""
    A, B, b = operands(layout)
    handle = StandIn()
    handle.refuse = True
    y = product(A, B, torch.tensor(b), layout, handle)
    y.sum().backward()
    assert (y == 0).all() and (A.grad == 0).all() and torch.isnan(B.grad).all()


@pytest.mark.parametrize("dtype,groups", [(torch.uint8, 255), (torch.uint8, 256), (torch.int8, 127), (torch.int8, 128),
                                          (torch.int8, 300), (torch.int16, 4096), (torch.int32, 256)])
def test_group_rows_of_narrow_indices(dtype, groups):
    """The count of groups need not fit into the indices' type."""
    expert = torch.tensor([3, 0, 120, 3, 126, 1]).to(dtype)
    order, offsets = experts.group_rows(expert, groups)
    assert order.tolist() == [1, 5, 0, 3, 2, 4]
    assert offsets.tolist() == [int((expert.long() < g).sum()) for g in range(groups)] + [6] and offsets.dtype == torch.int64
