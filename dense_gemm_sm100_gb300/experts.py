"""Expert products for torch models: row grouping and a differentiable
grouped product on the library's kernels.

``group_rows`` turns a router's choices into the row order and offsets that the
grouped products read (both stay on the device); ``grouped_matmul`` is
``Gemm.run_grouped`` with its two gradients.
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
    edges = torch.arange(groups + 1, device=expert.device, dtype=sorted_expert.dtype)
    return order, torch.searchsorted(sorted_expert, edges)


def _dense_rows(t: torch.Tensor) -> torch.Tensor:
    """t, or a copy when its rows overlap or are not unit-stride (an expanded
    gradient, a transposed view)."""
    ok = t.shape[-1] <= 1 or t.stride(-1) == 1
    for d in range(t.dim() - 1):
        ok = ok and (t.shape[d] <= 1 or t.stride(d) >= t.stride(d + 1) * t.shape[d + 1])
    return t if ok else t.contiguous()


class _GroupedMatmul(torch.autograd.Function):
    @staticmethod
    def forward(ctx, A, B, offsets, layout, dtype, out_dtype, handle):
        A, B = _dense_rows(A), _dense_rows(B)
        ctx.save_for_backward(A, B, offsets)
        ctx.config = (layout, dtype, handle)
        N = B.shape[2] if layout == _g.GEMM_B_ROW_MAJOR else B.shape[1]
        C = torch.zeros((A.shape[0], N), dtype=out_dtype, device=A.device)  # rows of no group give zeros
        return handle.run_grouped(A, B, offsets, C, layout, dtype)

    @staticmethod
    def backward(ctx, dC):
        A, B, offsets = ctx.saved_tensors
        layout, dtype, handle = ctx.config
        row = layout == _g.GEMM_B_ROW_MAJOR
        dC = _dense_rows(dC.to(A.dtype))
        dA = dB = None
        if ctx.needs_input_grad[0]:
            dA = torch.zeros_like(A, memory_format=torch.contiguous_format)
            handle.run_grouped(dC, B, offsets, dA, _g.GEMM_B_COL_MAJOR if row else _g.GEMM_B_ROW_MAJOR, dtype)
        if ctx.needs_input_grad[1]:
            dB = torch.empty_like(B, memory_format=torch.contiguous_format)
            left, right = (A, dC) if row else (dC, A)
            handle.run_grouped_wgrad(left, right, offsets, dB, dtype)
        return dA, dB, None, None, None, None, None


def grouped_matmul(A, B, offsets, layout_b="row", out_dtype=None, handle: _g.Gemm | None = None):
    """C[r] = A[r] · B[g] over row groups, differentiable in A and B.

    A is (rows, K) bfloat16, or float32 for the TF32 mode; B (groups, K, N), or
    (groups, N, K) with ``layout_b="col"``; offsets (groups + 1,) int64 on the
    device.  C has A's dtype unless ``out_dtype`` says otherwise (float32 for
    bfloat16 operands); rows of no group are zero.  The gradients have their
    operand's dtype, and dC enters the backward products in A's."""
    layout = _g.LAYOUTS.get(layout_b, layout_b)
    dtype = _g.GEMM_BF16 if A.dtype == torch.bfloat16 else _g.GEMM_TF32
    if A.device.type != "cuda":
        raise ValueError(f"A is on {A.device}: the grouped products run on a CUDA device")
    return _GroupedMatmul.apply(A, B, offsets, layout, dtype, out_dtype or A.dtype,
                                handle or _g._default_handle(A.device.index or 0))
