"""Expert products for torch models: row grouping and a differentiable
grouped product on the library's kernels.

``group_rows`` turns a router's choices into the row order and offsets that the
grouped products read (both stay on the device); ``grouped_matmul`` is
``Gemm.run_grouped`` with its two gradients, differentiable any number of times.
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
