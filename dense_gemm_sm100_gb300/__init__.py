"""GB300-native dense GEMM (C = A·B) behind a C ABI (include/gemm.h).

``dense_gemm_sm100_gb300.gemm`` is the Python binding, also of the grouped
expert products (include/gemm_grouped.h) and of microscaled 4-bit floating
point (include/gemm_mx4.h); ``experts`` makes the grouped product
differentiable for torch models; ``build`` compiles the CUDA library in-tree;
``inputs`` draws seeded operands; ``roofline`` holds the work/traffic model
used by the benchmark.
"""
from . import build, inputs, roofline  # noqa: F401
from .gemm import (GEMM_B_COL_MAJOR, GEMM_B_ROW_MAJOR, GEMM_BF16, GEMM_F32,  # noqa: F401
                   GEMM_TF32, Gemm, GemmError, GemmLibraryMissing, Mx4, default_handle, matmul,
                   mx4_empty)
