"""Expert products for torch models: routing, row grouping and a differentiable
grouped product on the library's kernels.

``route`` takes a router's logits to the chosen experts, their weights
(differentiable in the logits) and the row order and offsets that the grouped
products read, all on the device; ``group_rows`` makes the latter two from
choices made elsewhere; ``grouped_matmul`` is ``Gemm.run_grouped`` with its two
gradients, differentiable any number of times.
"""
from __future__ import annotations

import torch

from . import gemm as _g


def group_rows(expert: torch.Tensor, groups: int):
    """``(order, offsets)`` for a 1-D tensor of expert indices: ``order`` lists
    the rows sorted by expert (rows of one expert keep their order), and expert
    g owns ``order[offsets[g]:offsets[g + 1]]``."""
    if expert.dim() != 1:
        raise ValueError("expert must be 1-D")
    sorted_expert, order = torch.sort(expert, stable=True)
    if not expert.dtype.is_floating_point and torch.iinfo(expert.dtype).max < groups:
        sorted_expert = sorted_expert.long()  # 256 does not fit into a uint8 of 256 experts
    edges = torch.arange(groups + 1, device=expert.device, dtype=sorted_expert.dtype)
    return order, torch.searchsorted(sorted_expert, edges)


def _dense_rows(t: torch.Tensor) -> torch.Tensor:
    """t, or a copy when its rows overlap or are not unit-stride (an expanded
    gradient, a transposed view)."""
    if t.is_contiguous():
        return t
    ok = t.shape[-1] <= 1 or t.stride(-1) == 1
    for d in range(t.dim() - 1):
        ok = ok and (t.shape[d] <= 1 or t.stride(d) >= t.stride(d + 1) * t.shape[d + 1])
    return t if ok else t.contiguous()


def _product(A, B, offsets, layout, dtype, out_dtype, handle):
    # copies are taken out here, where autograd sees them
    return _dense_product(_dense_rows(A), _dense_rows(B), offsets, layout, dtype, out_dtype, handle)


def _dense_product(A, B, offsets, layout, dtype, out_dtype, handle):
    """A[r] · B[g], differentiable where autograd records (in a backward pass:
    with ``create_graph``; else the call skips autograd's bookkeeping, 20 to 30 us
    on the host)."""
    f = _GroupedMatmul.apply if torch.is_grad_enabled() else _run_product
    return f(A, B, offsets, layout, dtype, out_dtype, handle)


def _dense_outer(A, B, offsets, dtype, out_dtype, handle):
    """A_g^T · B_g, likewise."""
    f = _GroupedOuter.apply if torch.is_grad_enabled() else _run_outer
    return f(A, B, offsets, dtype, out_dtype, handle)


def _run_product(A, B, offsets, layout, dtype, out_dtype, handle):
    N = B.shape[2] if layout == _g.GEMM_B_ROW_MAJOR else B.shape[1]
    C = torch.zeros((A.shape[0], N), dtype=out_dtype, device=A.device)  # rows of no group give zeros
    return handle.run_grouped(A, B, offsets, C, layout, dtype)


def _run_outer(A, B, offsets, dtype, out_dtype, handle):
    C = torch.empty((offsets.shape[0] - 1, A.shape[1], B.shape[1]), dtype=out_dtype, device=A.device)
    return handle.run_grouped_wgrad(A, B, offsets, C, dtype, nan_on_error=True)


class _GroupedMatmul(torch.autograd.Function):
    """C[r] = A[r] · B[g], linear in A and in B.  Both gradients are grouped
    products again, taken through differentiable functions, so gradients of any
    order come out of the same two kernels."""

    @staticmethod
    def forward(ctx, A, B, offsets, layout, dtype, out_dtype, handle):
        ctx.save_for_backward(A, B, offsets)
        ctx.config = (layout, dtype, handle)
        return _run_product(A, B, offsets, layout, dtype, out_dtype, handle)

    @staticmethod
    def backward(ctx, dC):
        A, B, offsets = ctx.saved_tensors
        layout, dtype, handle = ctx.config
        row = layout == _g.GEMM_B_ROW_MAJOR
        dC = _dense_rows(dC.to(A.dtype))
        dA = dB = None
        if ctx.needs_input_grad[0]:
            flipped = _g.GEMM_B_COL_MAJOR if row else _g.GEMM_B_ROW_MAJOR
            dA = _dense_product(dC, B, offsets, flipped, dtype, A.dtype, handle)
        if ctx.needs_input_grad[1]:
            left, right = (A, dC) if row else (dC, A)
            dB = _dense_outer(left, right, offsets, dtype, B.dtype, handle)
        return dA, dB, None, None, None, None, None


class _GroupedOuter(torch.autograd.Function):
    """C[g] = A_g^T · B_g, the weight gradient, linear in A and in B."""

    @staticmethod
    def forward(ctx, A, B, offsets, dtype, out_dtype, handle):
        ctx.save_for_backward(A, B, offsets)
        ctx.config = (dtype, handle)
        return _run_outer(A, B, offsets, dtype, out_dtype, handle)

    @staticmethod
    def backward(ctx, dC):
        A, B, offsets = ctx.saved_tensors
        dtype, handle = ctx.config
        dC = _dense_rows(dC.to(A.dtype))
        dA = dB = None
        if ctx.needs_input_grad[0]:
            dA = _dense_product(B, dC, offsets, _g.GEMM_B_COL_MAJOR, dtype, A.dtype, handle)
        if ctx.needs_input_grad[1]:
            dB = _dense_product(A, dC, offsets, _g.GEMM_B_ROW_MAJOR, dtype, B.dtype, handle)
        return dA, dB, None, None, None, None


def grouped_matmul(A, B, offsets, layout_b="row", out_dtype=None, handle: _g.Gemm | None = None):
    """C[r] = A[r] · B[g] over row groups, differentiable in A and B.

    A is (rows, K) bfloat16, or float32 for the TF32 mode; B (groups, K, N), or
    (groups, N, K) with ``layout_b="col"``; offsets (groups + 1,) int64 on the
    device.  C has A's dtype unless ``out_dtype`` says otherwise (float32 for
    bfloat16 operands); rows of no group are zero.  The gradients have their
    operand's dtype, and dC enters the backward products in A's.  They are
    differentiable themselves (``create_graph=True``).

    Offsets that decrease or leave [0, rows] are found on the device: the output
    and dA are then zero, dB is NaN, and the handle's ``sync_status`` raises
    (``gemm.default_handle().sync_status()`` where no ``handle`` is given).
    The same call reports an expired wait inside a kernel, which leaves parts of
    the output and dA at zero and makes dB NaN until it has been reported.

    All calls run on torch's current stream; threads and streams may share a
    handle, the default one included."""
    layout = _g.LAYOUTS.get(layout_b, layout_b)
    dtype = _g.GEMM_BF16 if A.dtype == torch.bfloat16 else _g.GEMM_TF32
    if A.device.type != "cuda":
        raise ValueError(f"A is on {A.device}: the grouped products run on a CUDA device")
    return _product(A, B, offsets, layout, dtype, out_dtype or A.dtype,
                    handle or _g.default_handle(A.device.index or 0))


def _weights_of(logits, expert, scoring, renormalise, scale):
    """The weights of given choices as torch operations, for gradients of gradients."""
    chosen, x = expert >= 0, logits.float()
    index = expert.clamp(min=0)
    if scoring == "sigmoid":
        # a finite stand-in where there is no choice: 0 * nan would stay in the gradient
        score = torch.sigmoid(torch.gather(x, 1, index).masked_fill(~chosen, 0.0)).masked_fill(~chosen, 0.0)
        if renormalise:
            score = score / (score.sum(-1, keepdim=True) + 1e-20)
    elif renormalise:
        # finite in rows without any choice, below every logit in the others
        x = torch.gather(x, 1, index).masked_fill(~chosen, -float("inf"))
        x = x.masked_fill(~chosen.any(-1, keepdim=True), 0.0)
        score = torch.softmax(x, -1).masked_fill(~chosen, 0.0)
    else:
        x = x.masked_fill(~chosen.any(-1, keepdim=True), 0.0)
        score = torch.gather(torch.softmax(x, -1), 1, index).masked_fill(~chosen, 0.0)
    return scale * score


class _Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, k, scoring, bias, groups, top_groups, renormalise, scale, handle):
        out = _g.routing_empty(logits.shape[0], logits.shape[1], k, logits.device)
        handle.route(logits, out, scoring, bias, groups, top_groups, renormalise, scale)
        ctx.save_for_backward(logits, out.expert)
        ctx.config = (scoring, renormalise, scale, handle)
        ctx.mark_non_differentiable(out.expert, out.order, out.offsets)
        return tuple(out)

    @staticmethod
    def backward(ctx, dweights, *_):
        logits, expert = ctx.saved_tensors
        scoring, renormalise, scale, handle = ctx.config
        if torch.is_grad_enabled():  # create_graph
            w = _weights_of(logits, expert, scoring, renormalise, scale)
            dlogits, = torch.autograd.grad(w, logits, dweights, create_graph=True)
        else:
            dlogits = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
            handle.route_grad(logits, expert, dweights.contiguous(), dlogits, scoring, renormalise, scale)
        return (dlogits,) + (None,) * 8


def route(logits, k, scoring="softmax", bias=None, groups=1, top_groups=1, renormalise=True, scale=1.0,
          handle: _g.Gemm | None = None) -> _g.Routing:
    """The k experts of every row of ``logits`` (tokens, experts), their weights,
    and the rows token * k + choice sorted by expert: ``Gemm.route`` with
    ``weights`` differentiable in the logits (any number of times; the choices
    are constants, and so is ``bias``).

    With ``r = route(logits, k)`` and ``rows = x[r.order // k]``, expert g's rows
    are ``rows[r.offsets[g]:r.offsets[g + 1]]``, as ``grouped_matmul`` takes them.
    Logits of minus infinity are never chosen; choices that are not there
    (``expert`` -1, weight 0) come first in ``order``, in no expert's rows."""
    if logits.device.type != "cuda":
        raise ValueError(f"logits are on {logits.device}: the router runs on a CUDA device")
    if logits.dim() != 2:
        raise ValueError("logits must be 2-D")
    h = handle or _g.default_handle(logits.device.index or 0)
    return _g.Routing(*_Route.apply(_dense_rows(logits), k, scoring, None if bias is None else bias.detach(), groups,
                                    top_groups, renormalise, scale, h))
