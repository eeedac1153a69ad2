"""Python binding of the C ABI in include/gemm.h (argument marshalling only).

The functions ``gemm_create``, ``gemm_run``, ``gemm_run_host``,
``gemm_destroy``, ``gemm_validate``, ``gemm_sync_status``,
``gemm_set_option``, ``gemm_last_error_string``, ``gemm_status_string``,
``gemm_last_path``, ``gemm_launch_count``, ``gemm_version``,
``gemm_run_noalloc``, ``gemm_ladder_run``, ``gemm_ladder_name``,
``gemm_peak_fma_run`` and ``gemm_peak_mma_run``, and those of
include/gemm_grouped.h, include/gemm_mx4.h, include/gemm_i8.h,
include/gemm_route.h and include/gemm_ortho.h, take and return the same plain
values as their C counterparts (pointers as ints; the FLOP-count out-parameter
of the peak calls is returned as a second value).  ``Gemm`` wraps a handle for torch tensors;
``Mx4`` holds a matrix in microscaled 4-bit floating point, ``I8`` one in 8-bit
integers, ``Routing`` the choices of a router.  Every GEMM step runs in the library's CUDA
kernels; there is no other code path, and calling anything here without the
built library raises ``GemmLibraryMissing``.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Any, NamedTuple

from . import build as _build

GEMM_B_ROW_MAJOR = 0
GEMM_B_COL_MAJOR = 1
GEMM_F32 = 0
GEMM_TF32 = 1
GEMM_BF16 = 2
GEMM_F32_3XTF32 = 3

GEMM_OK = 0
GEMM_ERR_INVALID = -1
GEMM_ERR_ALIGNMENT = -2
GEMM_ERR_CUDA = -3
GEMM_ERR_TIMEOUT = -4
GEMM_ERR_DEVICE = -5
GEMM_ERR_NOMEM = -6

GEMM_OPT_FORCE_REPACK = 1
GEMM_OPT_WAIT_TIMEOUT_NS = 2
GEMM_OPT_SIMT_GROUP_M = 3
GEMM_OPT_TC_GROUP_M = 4
GEMM_OPT_MAX_CTAS = 5
GEMM_OPT_SIMT_CONFIG = 6
GEMM_OPT_SPLIT_K = 7
GEMM_OPT_TC_CLUSTER = 8
GEMM_OPT_TC_TMA_STORE = 9
GEMM_OPT_DEBUG_DROP_LOAD = 10
GEMM_OPT_ELEMENTWISE = 11
GEMM_OPT_WORKSPACE_LIMIT = 12
GEMM_OPT_TC_STAGE_SLICES = 13
GEMM_OPT_STREAM_K = 14
GEMM_OPT_SIMT_SMALL = 15
GEMM_OPT_GROUPED_TILE = 16
GEMM_OPT_ORTHO_TILE = 17

GEMM_GROUPED_MAX_GROUPS = 4096
GEMM_GROUPED_NAN_ON_ERROR = 0x100
GEMM_MX4_BLOCK = 32

GEMM_ROUTE_MAX_EXPERTS = 1024
GEMM_ROUTE_MAX_K = 31
GEMM_ROUTE_MAX_GROUPS = 32
GEMM_ROUTE_SIGMOID = 1
GEMM_ROUTE_RENORMALISE = 2

GEMM_ORTHO_MAX_STEPS = 32

DTYPES = {"f32": GEMM_F32, "tf32": GEMM_TF32, "bf16": GEMM_BF16, "f32x3": GEMM_F32_3XTF32}
LAYOUTS = {"row": GEMM_B_ROW_MAJOR, "col": GEMM_B_COL_MAJOR}

LIB_PATH = _build.LIB_PATH


class GemmLibraryMissing(RuntimeError):
    """The CUDA library has not been built (run ``__graft_entry__.build()``)."""


class GemmError(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(f"{gemm_status_string(code)}: {message}")
        self.code = code


_lock = threading.Lock()
_lib = None


def load_library():
    """Load ``libdense_gemm_gb300.so`` (raises GemmLibraryMissing if absent)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise GemmLibraryMissing(
                f"{LIB_PATH} is missing: build the CUDA library first "
                "(python -c 'import __graft_entry__ as g; g.build()')")
        lib = ctypes.CDLL(LIB_PATH)
        i64, vp, ci = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
        run_args = [vp, ci, i64, i64, i64, vp, i64, vp, i64, vp, i64, ci, vp]
        sig = {
            "gemm_create": ([ctypes.POINTER(vp), ci], ci),
            "gemm_destroy": ([vp], ci),
            "gemm_run": (run_args, ci),
            "gemm_run_host": (run_args, ci),
            "gemm_validate": ([ci, i64, i64, i64, vp, i64, vp, i64, vp, i64, ci], ci),
            "gemm_sync_status": ([vp, vp], ci),
            "gemm_set_option": ([vp, ci, i64], ci),
            "gemm_last_error_string": ([vp], ctypes.c_char_p),
            "gemm_status_string": ([ci], ctypes.c_char_p),
            "gemm_last_path": ([vp], ctypes.c_char_p),
            "gemm_launch_count": ([vp], i64),
            "gemm_version": ([], ci),
            "gemm_run_noalloc": ([ci, i64, i64, i64, vp, i64, vp, i64, vp, i64, ci, vp], ci),
            "gemm_noalloc_sync_status": ([vp], ci),
            "gemm_noalloc_set_option": ([ci, i64], ci),
            "gemm_ladder_run": ([ci, i64, i64, i64, vp, vp, vp, vp], ci),
            "gemm_ladder_name": ([ci], ctypes.c_char_p),
            "gemm_peak_fma_run": ([ci, i64, vp, vp, ctypes.POINTER(ctypes.c_double)], ci),
            "gemm_peak_mma_run": ([ci, i64, vp, ctypes.c_uint64, vp, ctypes.POINTER(ctypes.c_double)], ci),
        }
        grouped = [ci, i64, i64, i64, i64, vp, vp, i64, vp, i64, i64, vp, i64, ci, ci]
        wgrad = [i64, i64, i64, i64, vp, vp, i64, vp, i64, vp, i64, i64, ci, ci]
        quantise = [ci, i64, i64, i64, vp, i64, i64, ci, vp, i64, vp, i64]
        dequantise = [i64, i64, vp, i64, vp, i64, vp, i64, ci]
        mx4 = [i64, i64, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, ci]
        mx4_grouped = [i64, i64, i64, i64, vp, vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, ci]
        sig.update({
            "gemm_grouped_run": ([vp, *grouped, vp], ci),
            "gemm_grouped_wgrad": ([vp, *wgrad, vp], ci),
            "gemm_grouped_validate": (grouped, ci),
            "gemm_grouped_wgrad_validate": (wgrad, ci),
            "gemm_mx4_code_pitch": ([i64], i64),
            "gemm_mx4_scale_pitch": ([i64], i64),
            "gemm_mx4_quantise": ([vp, *quantise, vp], ci),
            "gemm_mx4_dequantise": ([vp, *dequantise, vp], ci),
            "gemm_mx4_run": ([vp, *mx4, vp], ci),
            "gemm_mx4_grouped_run": ([vp, *mx4_grouped, vp], ci),
            "gemm_mx4_quantise_validate": (quantise, ci),
            "gemm_mx4_dequantise_validate": (dequantise, ci),
            "gemm_mx4_validate": (mx4_grouped, ci),
        })
        i8_quantise = [ci, i64, i64, i64, vp, i64, i64, ci, vp, i64, vp]
        i8_dequantise = [i64, i64, vp, i64, vp, vp, i64, ci]
        i8 = [i64, i64, i64, vp, i64, vp, vp, i64, vp, vp, i64, ci]
        i8_grouped = [i64, i64, i64, i64, vp, vp, i64, vp, vp, i64, vp, vp, i64, ci]
        sig.update({
            "gemm_i8_code_pitch": ([i64], i64),
            "gemm_i8_quantise": ([vp, *i8_quantise, vp], ci),
            "gemm_i8_dequantise": ([vp, *i8_dequantise, vp], ci),
            "gemm_i8_run": ([vp, *i8, vp], ci),
            "gemm_i8_grouped_run": ([vp, *i8_grouped, vp], ci),
            "gemm_i8_quantise_validate": (i8_quantise, ci),
            "gemm_i8_dequantise_validate": (i8_dequantise, ci),
            "gemm_i8_validate": (i8_grouped, ci),
        })
        cf = ctypes.c_float
        route = [i64, i64, i64, vp, i64, ci, vp, i64, i64, ci, cf, vp, vp, vp, vp]
        route_grad = [i64, i64, i64, vp, i64, ci, vp, vp, ci, cf, vp, i64]
        sig.update({
            "gemm_route": ([vp, *route, vp], ci),
            "gemm_route_grad": ([vp, *route_grad, vp], ci),
            "gemm_route_validate": (route, ci),
            "gemm_route_grad_validate": (route_grad, ci),
        })
        ortho = [i64, i64, i64, vp, i64, i64, vp, i64, i64, ci, ci, vp, cf]
        sig.update({
            "gemm_orthogonalise": ([vp, *ortho, vp], ci),
            "gemm_orthogonalise_validate": (ortho, ci),
        })
        for name, (argtypes, restype) in sig.items():
            fn = getattr(lib, name)
            fn.argtypes = argtypes
            fn.restype = restype
        _lib = lib
        return lib


# ----------------------------------------------------------- C-named functions

def gemm_version() -> int:
    return load_library().gemm_version()


def gemm_status_string(code: int) -> str:
    return load_library().gemm_status_string(code).decode()


def gemm_create(device: int = 0) -> int:
    h = ctypes.c_void_p()
    rc = load_library().gemm_create(ctypes.byref(h), device)
    if rc != GEMM_OK:
        raise GemmError(rc, f"gemm_create(device={device}) failed")
    return h.value


def gemm_destroy(handle: int) -> int:
    return load_library().gemm_destroy(handle)


def gemm_run(handle, layout_b, M, N, K, A, lda, B, ldb, C, ldc, dtype, stream) -> int:
    return load_library().gemm_run(handle, layout_b, M, N, K, A, lda, B, ldb, C, ldc, dtype, stream)


def gemm_run_host(handle, layout_b, M, N, K, A, lda, B, ldb, C, ldc, dtype, stream) -> int:
    return load_library().gemm_run_host(handle, layout_b, M, N, K, A, lda, B, ldb, C, ldc,
                                        dtype, stream)


def gemm_validate(layout_b, M, N, K, A, lda, B, ldb, C, ldc, dtype) -> int:
    return load_library().gemm_validate(layout_b, M, N, K, A, lda, B, ldb, C, ldc, dtype)


def gemm_sync_status(handle, stream) -> int:
    return load_library().gemm_sync_status(handle, stream)


def gemm_set_option(handle, option, value) -> int:
    return load_library().gemm_set_option(handle, option, value)


def gemm_last_error_string(handle) -> str:
    return load_library().gemm_last_error_string(handle).decode()


def gemm_last_path(handle) -> str:
    return load_library().gemm_last_path(handle).decode()


def gemm_launch_count(handle) -> int:
    return load_library().gemm_launch_count(handle)


def gemm_run_noalloc(layout_b, M, N, K, A, lda, B, ldb, C, ldc, dtype, stream) -> int:
    """C = A·B with no device allocation (no handle; the current device's
    static scratch holds re-packed operands, at most
    GEMM_NOALLOC_SCRATCH_BYTES).  For callers that cannot allocate."""
    return load_library().gemm_run_noalloc(layout_b, M, N, K, A, lda, B, ldb, C, ldc, dtype,
                                           stream)


def gemm_noalloc_sync_status(stream) -> int:
    """Waits for `stream`; GEMM_ERR_TIMEOUT if an in-kernel wait of an
    allocation-free call on the current device expired (then cleared)."""
    return load_library().gemm_noalloc_sync_status(stream)


def gemm_noalloc_set_option(option, value) -> int:
    """Process-wide wait limit / test hook of the allocation-free calls."""
    return load_library().gemm_noalloc_set_option(option, value)


# include/gemm_grouped.h and include/gemm_mx4.h, argument for argument.

def gemm_grouped_run(*args) -> int:
    return load_library().gemm_grouped_run(*args)


def gemm_grouped_wgrad(*args) -> int:
    return load_library().gemm_grouped_wgrad(*args)


def gemm_grouped_validate(*args) -> int:
    return load_library().gemm_grouped_validate(*args)


def gemm_grouped_wgrad_validate(*args) -> int:
    return load_library().gemm_grouped_wgrad_validate(*args)


def gemm_mx4_code_pitch(K) -> int:
    return load_library().gemm_mx4_code_pitch(K)


def gemm_mx4_scale_pitch(K) -> int:
    return load_library().gemm_mx4_scale_pitch(K)


def gemm_mx4_quantise(*args) -> int:
    return load_library().gemm_mx4_quantise(*args)


def gemm_mx4_dequantise(*args) -> int:
    return load_library().gemm_mx4_dequantise(*args)


def gemm_mx4_run(*args) -> int:
    return load_library().gemm_mx4_run(*args)


def gemm_mx4_grouped_run(*args) -> int:
    return load_library().gemm_mx4_grouped_run(*args)


def gemm_mx4_quantise_validate(*args) -> int:
    return load_library().gemm_mx4_quantise_validate(*args)


def gemm_mx4_dequantise_validate(*args) -> int:
    return load_library().gemm_mx4_dequantise_validate(*args)


def gemm_mx4_validate(*args) -> int:
    return load_library().gemm_mx4_validate(*args)


# include/gemm_i8.h, include/gemm_route.h and include/gemm_ortho.h, argument for
# argument.

def gemm_i8_code_pitch(K) -> int:
    return load_library().gemm_i8_code_pitch(K)


def gemm_i8_quantise(*args) -> int:
    return load_library().gemm_i8_quantise(*args)


def gemm_i8_dequantise(*args) -> int:
    return load_library().gemm_i8_dequantise(*args)


def gemm_i8_run(*args) -> int:
    return load_library().gemm_i8_run(*args)


def gemm_i8_grouped_run(*args) -> int:
    return load_library().gemm_i8_grouped_run(*args)


def gemm_i8_quantise_validate(*args) -> int:
    return load_library().gemm_i8_quantise_validate(*args)


def gemm_i8_dequantise_validate(*args) -> int:
    return load_library().gemm_i8_dequantise_validate(*args)


def gemm_i8_validate(*args) -> int:
    return load_library().gemm_i8_validate(*args)


def gemm_route(*args) -> int:
    return load_library().gemm_route(*args)


def gemm_route_grad(*args) -> int:
    return load_library().gemm_route_grad(*args)


def gemm_route_validate(*args) -> int:
    return load_library().gemm_route_validate(*args)


def gemm_route_grad_validate(*args) -> int:
    return load_library().gemm_route_grad_validate(*args)


def gemm_orthogonalise(*args) -> int:
    return load_library().gemm_orthogonalise(*args)


def gemm_orthogonalise_validate(*args) -> int:
    return load_library().gemm_orthogonalise_validate(*args)


GEMM_NOALLOC_SCRATCH_BYTES = 64 * 1024 * 1024

# Labelled benchmark suite (include/gemm_ladder.h): the pages' optimisation
# ladder and the PMPP worked kernels.  Not the library's GEMM path.
GEMM_LADDER_STEPS = {1: "naive", 2: "smem_tiling", 3: "thread_tiling", 4: "vectorized",
                     5: "conflict_free", 6: "warp_tiling", 7: "double_buffer", 8: "cp_async"}
GEMM_LADDER_PMPP_CORNER_TURN = 101
GEMM_LADDER_PMPP_COARSENED = 102


def gemm_ladder_run(step, M, N, K, A, B, C, stream) -> int:
    return load_library().gemm_ladder_run(step, M, N, K, A, B, C, stream)


def gemm_ladder_name(step) -> str:
    return load_library().gemm_ladder_name(step).decode()


# Peak-rate microbenchmarks (include/gemm_peaks.h): the compute roofs.

def gemm_peak_fma_run(packed, iters, sink, stream) -> tuple[int, float]:
    flops = ctypes.c_double(0.0)
    rc = load_library().gemm_peak_fma_run(packed, iters, sink, stream, ctypes.byref(flops))
    return rc, flops.value


def gemm_peak_mma_run(dtype, iters, status, timeout_ns, stream) -> tuple[int, float]:
    flops = ctypes.c_double(0.0)
    rc = load_library().gemm_peak_mma_run(dtype, iters, status, timeout_ns, stream, ctypes.byref(flops))
    return rc, flops.value


def measure_peak(kind: str, iters: int, reps: int = 3, stream=None) -> dict:
    """Time the microbenchmark `kind` ("ffma", "ffma2", "mma_bf16",
    "mma_tf32") with CUDA events on `stream`: one warm-up launch, then the
    best of `reps` launches.  Returns TFLOP/s and the launch time."""
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    sh = _stream_handle(s)
    sink = torch.zeros(2, dtype=torch.float32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def launch():
        if kind in ("ffma", "ffma2"):
            rc, fl = gemm_peak_fma_run(1 if kind == "ffma2" else 0, iters, sink.data_ptr(), sh)
        else:
            dt = GEMM_BF16 if kind == "mma_bf16" else GEMM_TF32
            rc, fl = gemm_peak_mma_run(dt, iters, status.data_ptr(), 0, sh)
        if rc != GEMM_OK:
            raise GemmError(rc, f"{kind} microbenchmark: {gemm_status_string(rc)}")
        return fl

    launch()
    best_ms, flops = None, 0.0
    for _ in range(reps):
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        e0.record(s)
        flops = launch()
        e1.record(s)
        e1.synchronize()
        ms = e0.elapsed_time(e1)
        best_ms = ms if best_ms is None else min(best_ms, ms)
    if int(status.item()) != 0:
        raise GemmError(GEMM_ERR_TIMEOUT, f"{kind} microbenchmark: a wait expired")
    return {"tflops": flops / (best_ms * 1e-3) / 1e12, "ms": best_ms, "flops": flops}


# ------------------------------------------------------------- torch wrapper

def _stream_handle(stream) -> int:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


# Argument marshalling of the grouped and 4-bit calls.  These run per call, in
# front of kernels of a few microseconds, so each looks at a tensor's fields
# once and nothing is imported or locked on the way.

_float_codes = None


def _type_code(t, name):
    global _float_codes
    if _float_codes is None:
        import torch
        _float_codes = {torch.float32: GEMM_F32, torch.bfloat16: GEMM_BF16}
    code = _float_codes.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be float32 or bfloat16, not {t.dtype}")
    return code


def _on_device(t, name, device):
    if not t.is_cuda or t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, the handle on cuda:{device}")


def _matrix(t, name, device):
    """(rows, columns, pitch, type code) of a 2-D operand on `device`."""
    _on_device(t, name, device)
    shape, stride = t.shape, t.stride()
    if len(shape) != 2:
        raise ValueError(f"{name} must be 2-D")
    rows, cols = shape
    if cols > 1 and stride[1] != 1:
        raise ValueError(f"{name} must have unit stride along rows")
    ld = cols if cols > 0 else 1
    if rows > 1:
        if stride[0] < cols:
            raise ValueError(f"the rows of {name} overlap")
        if stride[0] > ld:
            ld = stride[0]
    return rows, cols, ld, _type_code(t, name)


def _matrices(t, name, device):
    """(matrices, rows, columns, pitch, matrix stride, type code) of a 3-D one."""
    _on_device(t, name, device)
    shape, stride = t.shape, t.stride()
    if len(shape) != 3:
        raise ValueError(f"{name} must be 3-D, matrices first")
    n, rows, cols = shape
    if cols > 1 and stride[2] != 1:
        raise ValueError(f"{name} must have unit stride along rows")
    ld = cols if cols > 0 else 1
    if rows > 1:
        if stride[1] < cols:
            raise ValueError(f"the rows of {name} overlap")
        if stride[1] > ld:
            ld = stride[1]
    return n, rows, cols, ld, (stride[0] if n > 1 else rows * ld), _type_code(t, name)


_int64 = None


def _offsets(t, groups, device):
    global _int64
    if _int64 is None:
        import torch
        _int64 = torch.int64
    _on_device(t, "offsets", device)
    if t.dtype != _int64 or t.dim() != 1 or t.shape[0] != groups + 1 or (groups > 0 and t.stride(0) != 1):
        raise ValueError(f"offsets must be a contiguous int64 tensor of {groups + 1} values")
    return t.data_ptr()


def _operand_types(dt, a, b):
    want = GEMM_BF16 if dt == GEMM_BF16 else GEMM_F32
    if a != want or b != want:
        raise ValueError(f"A and B must be {'bfloat16' if dt == GEMM_BF16 else 'float32'} for this dtype")


_current_raw_stream = None


def _raw_stream(stream, device):
    """The caller's stream, or torch's current one on `device`, as a pointer."""
    global _current_raw_stream
    if stream is not None:
        return _stream_handle(stream)
    if _current_raw_stream is None:
        import torch
        _current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda d: torch.cuda.current_stream(d).cuda_stream)
    return _current_raw_stream(device)


class Mx4:
    """A matrix of rows x K elements in microscaled 4-bit floating point.

    ``codes`` (rows x pitch bytes, two E2M1 codes a byte, the even element in
    the low half) and ``scales`` (rows x pitch bytes, one E8M0 byte per 32
    elements) are uint8 tensors; rows and pitches are multiples of 16 bytes
    (``mx4_empty`` makes them so).  The expert matrices of a grouped product
    follow one another along the rows."""

    def __init__(self, codes, scales, K: int):
        import torch
        blocks = -(-K // GEMM_MX4_BLOCK)
        for name, t, need in (("codes", codes, blocks * 16), ("scales", scales, blocks)):
            if t.dtype != torch.uint8 or t.dim() != 2:
                raise ValueError(f"{name} must be a 2-D uint8 tensor")
            if t.shape[1] < need or (t.shape[1] > 1 and t.stride(1) != 1):
                raise ValueError(f"{name} must hold {need} bytes of each row, next to one another")
        if codes.shape[0] != scales.shape[0] or codes.device != scales.device:
            raise ValueError("codes and scales must have the same rows and device")
        self.codes, self.scales, self.K = codes, scales, int(K)
        self.rows = codes.shape[0]
        self._pitches = [t.stride(0) if self.rows > 1 else t.shape[1] for t in (codes, scales)]
        if self.rows > 1 and (codes.stride(0) < blocks * 16 or scales.stride(0) < blocks):
            raise ValueError("the rows of codes or scales overlap")
        self._device = codes.get_device() if codes.is_cuda else None

    @property
    def device(self):
        return self.codes.device

    def _args(self, device):
        if self._device != device:
            raise ValueError(f"a 4-bit operand is on {self.device}, the handle on cuda:{device}")
        return self.codes.data_ptr(), self._pitches[0], self.scales.data_ptr(), self._pitches[1]


def mx4_empty(rows: int, K: int, device="cuda") -> Mx4:
    """Uninitialised ``Mx4`` storage for rows x K elements."""
    import torch
    return Mx4(torch.empty((rows, gemm_mx4_code_pitch(K)), dtype=torch.uint8, device=device),
               torch.empty((rows, gemm_mx4_scale_pitch(K)), dtype=torch.uint8, device=device), K)


class I8:
    """A matrix of rows x K elements in 8-bit integers with a scale a row.

    ``codes`` is (rows, pitch) int8, rows and pitch multiples of 16 bytes
    (``i8_empty`` makes them so), ``scales`` (rows,) float32.  The expert matrices
    of a grouped product follow one another along the rows."""

    def __init__(self, codes, scales, K: int):
        import torch
        if codes.dtype != torch.int8 or codes.dim() != 2:
            raise ValueError("codes must be a 2-D int8 tensor")
        if codes.shape[1] < K or (codes.shape[1] > 1 and codes.stride(1) != 1):
            raise ValueError(f"codes must hold {K} bytes of each row, next to one another")
        if scales.dtype != torch.float32 or scales.dim() != 1 or not scales.is_contiguous():
            raise ValueError("scales must be a contiguous 1-D float32 tensor")
        if codes.shape[0] != scales.shape[0] or codes.device != scales.device:
            raise ValueError("codes and scales must have the same rows and device")
        self.codes, self.scales, self.K = codes, scales, int(K)
        self.rows = codes.shape[0]
        self._pitch = codes.stride(0) if self.rows > 1 else codes.shape[1]
        if self._pitch < K:
            raise ValueError("the rows of codes overlap")
        self._device = codes.get_device() if codes.is_cuda else None

    @property
    def device(self):
        return self.codes.device

    def _args(self, device):
        if self._device != device:
            raise ValueError(f"an 8-bit operand is on {self.device}, the handle on cuda:{device}")
        return self.codes.data_ptr(), self._pitch, self.scales.data_ptr()


def i8_empty(rows: int, K: int, device="cuda") -> I8:
    """Uninitialised ``I8`` storage for rows x K elements."""
    import torch
    return I8(torch.empty((rows, gemm_i8_code_pitch(K)), dtype=torch.int8, device=device),
              torch.empty(rows, dtype=torch.float32, device=device), K)


class Routing(NamedTuple):
    """A router's choices: ``weights`` (tokens, k) float32 and ``expert``
    (tokens, k) int64, -1 where there is none; ``order`` (tokens * k,) int64, the
    rows token * k + choice sorted by expert, and ``offsets`` (experts + 1,)
    int64, the experts' bounds in it."""

    weights: Any
    expert: Any
    order: Any
    offsets: Any


def routing_empty(tokens: int, experts: int, k: int, device="cuda") -> Routing:
    """Uninitialised ``Routing`` storage."""
    import torch
    ints = lambda *shape: torch.empty(shape, dtype=torch.int64, device=device)
    return Routing(torch.empty((tokens, k), dtype=torch.float32, device=device), ints(tokens, k), ints(tokens * k),
                   ints(experts + 1))


_plain_types = None


def _plain(t, name, shape, kind, device):
    """The address of a contiguous tensor of the given shape; kind "int64" or "float32"."""
    global _plain_types
    if _plain_types is None:
        import torch
        _plain_types = {"int64": torch.int64, "float32": torch.float32}
    _on_device(t, name, device)
    if t.dtype != _plain_types[kind] or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {kind} tensor of shape {shape}")
    return t.data_ptr()


def _route_flags(scoring, renormalise):
    if scoring not in ("softmax", "sigmoid"):
        raise ValueError(f"scoring must be 'softmax' or 'sigmoid', not {scoring!r}")
    return (GEMM_ROUTE_SIGMOID if scoring == "sigmoid" else 0) | (GEMM_ROUTE_RENORMALISE if renormalise else 0)


def _step_table(steps, coefficients):
    """The C table of 3 * steps coefficients."""
    if steps < 1 or steps > GEMM_ORTHO_MAX_STEPS:
        raise ValueError(f"steps must be in 1..{GEMM_ORTHO_MAX_STEPS}")
    rows = coefficients if hasattr(coefficients[0], "__len__") else [coefficients] * steps
    if len(rows) != steps or any(len(r) != 3 for r in rows):
        raise ValueError("coefficients must be three numbers, or three for every step")
    return (ctypes.c_float * (3 * steps))(*(float(v) for r in rows for v in r))


class Gemm:
    """A library handle used with torch tensors.

    ``run(A, B, C, layout_b, dtype)`` computes C = A·B on the GPU: A is (M, K)
    row-major, B is (K, N) for ``layout_b="row"`` or (N, K) for ``"col"``
    (each row holding one column of the logical B), C is (M, N).  Rows may be
    padded (any stride(0) >= columns, stride(1) == 1).  The call is queued on
    ``stream`` (default: torch's current stream) and returns at once.  Calls of
    several host threads take turns.
    """

    def __init__(self, device: int = 0):
        self.device = device
        self.handle = gemm_create(device)
        self._lib = load_library()
        self._turn = threading.Lock()  # the library wants one thread at a time on a handle

    def close(self):
        if self.handle:
            gemm_destroy(self.handle)
            self.handle = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _check(self, rc: int):
        if rc != GEMM_OK:
            raise GemmError(rc, gemm_last_error_string(self.handle))

    def set_option(self, option: int, value: int):
        with self._turn:
            self._check(gemm_set_option(self.handle, option, int(value)))

    @staticmethod
    def _dims(A, B, layout_b):
        M, K = A.shape
        if layout_b == GEMM_B_ROW_MAJOR:
            Kb, N = B.shape
        else:
            N, Kb = B.shape
        if Kb != K:
            raise ValueError(f"inner dimensions differ: A has K={K}, B has K={Kb}")
        return M, N, K

    @staticmethod
    def _ld(t):
        if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
            raise ValueError("operands must be 2-D with unit stride along rows")
        if t.shape[0] > 1 and t.stride(0) < t.shape[1]:
            raise ValueError("the rows of an operand overlap")
        return max(t.stride(0), t.shape[1], 1)

    def run(self, A, B, C, layout_b="row", dtype="f32", stream=None):
        lb = LAYOUTS.get(layout_b, layout_b)
        dt = DTYPES.get(dtype, dtype)
        M, N, K = self._dims(A, B, lb)
        if tuple(C.shape) != (M, N):
            raise ValueError(f"C has shape {tuple(C.shape)}, expected {(M, N)}")
        with self._turn:
            self._check(gemm_run(self.handle, lb, M, N, K, A.data_ptr(), self._ld(A), B.data_ptr(),
                                 self._ld(B), C.data_ptr(), self._ld(C), dt, _stream_handle(stream)))
        return C

    def run_host(self, A, B, C, layout_b="row", dtype="f32", stream=None):
        """As ``run`` with CPU tensors (pinned for asynchronous copies): the
        library copies A and B in, runs, and copies C out on ``stream``."""
        lb = LAYOUTS.get(layout_b, layout_b)
        dt = DTYPES.get(dtype, dtype)
        M, N, K = self._dims(A, B, lb)
        with self._turn:
            self._check(gemm_run_host(self.handle, lb, M, N, K, A.data_ptr(), self._ld(A),
                                      B.data_ptr(), self._ld(B), C.data_ptr(), self._ld(C), dt,
                                      _stream_handle(stream)))
        return C

    def run_grouped(self, A, B, offsets, C, layout_b="row", dtype="bf16", stream=None):
        """C[r] = A[r] · B[g] for the rows r of every group g.

        A is (rows, K) with the rows sorted by group, ``offsets`` (groups + 1,)
        int64 on the device, B (groups, K, N) for ``layout_b="row"`` or
        (groups, N, K) for ``"col"``, C (rows, N) float32 or bfloat16.  Rows
        outside [offsets[0], offsets[-1]) keep what C held.  ``dtype`` is
        "bf16" or "tf32"."""
        lb = LAYOUTS.get(layout_b, layout_b)
        dt = DTYPES.get(dtype, dtype)
        dev = self.device
        M, K, lda, a_type = _matrix(A, "A", dev)
        rows, N, ldc, c_type = _matrix(C, "C", dev)
        groups, d1, d2, ldb, stride_b, b_type = _matrices(B, "B", dev)
        Kb, Nb = (d1, d2) if lb == GEMM_B_ROW_MAJOR else (d2, d1)
        if Kb != K or Nb != N or rows != M:
            raise ValueError(f"shapes differ: A {tuple(A.shape)}, B {tuple(B.shape)} ({layout_b}), C {tuple(C.shape)}")
        _operand_types(dt, a_type, b_type)
        with self._turn:
            rc = self._lib.gemm_grouped_run(self.handle, lb, groups, M, N, K, _offsets(offsets, groups, dev),
                                            A.data_ptr(), lda, B.data_ptr(), ldb, stride_b, C.data_ptr(), ldc, dt,
                                            c_type, _raw_stream(stream, dev))
            if rc:
                self._check(rc)
        return C

    def run_grouped_wgrad(self, A, B, offsets, C, dtype="bf16", stream=None, nan_on_error=False):
        """C[g] = A_g^T · B_g over the rows of group g (zeros where it has none).

        A is (rows, M), B (rows, N), C (groups, M, N) float32 or bfloat16: the
        gradient of a row-major weight with A the input and B the output's
        gradient, of a column-major weight with the two exchanged.
        ``nan_on_error``: C is NaN where the offsets are refused (else it keeps
        what it held), and while an expired wait of the handle is unreported."""
        dt = DTYPES.get(dtype, dtype)
        dev = self.device
        rows, M, lda, a_type = _matrix(A, "A", dev)
        rows_b, N, ldb, b_type = _matrix(B, "B", dev)
        groups, Mc, Nc, ldc, stride_c, c_type = _matrices(C, "C", dev)
        if rows_b != rows or Mc != M or Nc != N:
            raise ValueError(f"shapes differ: A {tuple(A.shape)}, B {tuple(B.shape)}, C {tuple(C.shape)}")
        _operand_types(dt, a_type, b_type)
        with self._turn:
            rc = self._lib.gemm_grouped_wgrad(self.handle, groups, rows, M, N, _offsets(offsets, groups, dev),
                                              A.data_ptr(), lda, B.data_ptr(), ldb, C.data_ptr(), ldc, stride_c, dt,
                                              c_type | (GEMM_GROUPED_NAN_ON_ERROR if nan_on_error else 0),
                                              _raw_stream(stream, dev))
            if rc:
                self._check(rc)
        return C

    def route(self, logits, out: Routing, scoring="softmax", bias=None, groups=1, top_groups=1, renormalise=True,
              scale=1.0, stream=None):
        """Every token's k experts and their weights, and the rows sorted by
        expert, into ``out`` (k is the width of ``out.expert``).

        logits is (tokens, experts) float32 or bfloat16; ``bias`` (experts,)
        float32 is added to the scores for the choice alone; of ``groups``
        equal groups of neighbouring experts the ``top_groups`` best by the sum
        of their two best experts stay open.  Weights are the scores
        ("softmax" or "sigmoid"), renormalised over the choices or not, times
        ``scale``.  Logits of minus infinity are never chosen."""
        dev = self.device
        T, E, ld, l_type = _matrix(logits, "logits", dev)
        if out.expert.dim() != 2:
            raise ValueError("out.expert must be 2-D")
        k = out.expert.shape[1]
        flags = _route_flags(scoring, renormalise)
        weights = _plain(out.weights, "out.weights", (T, k), "float32", dev)
        expert = _plain(out.expert, "out.expert", (T, k), "int64", dev)
        order = _plain(out.order, "out.order", (T * k,), "int64", dev)
        offsets = _plain(out.offsets, "out.offsets", (E + 1,), "int64", dev)
        b = None if bias is None else _plain(bias, "bias", (E,), "float32", dev)
        with self._turn:
            rc = self._lib.gemm_route(self.handle, T, E, k, logits.data_ptr(), ld, l_type, b, groups, top_groups, flags,
                                      scale, weights, expert, order, offsets, _raw_stream(stream, dev))
            if rc:
                self._check(rc)
        return out

    def route_grad(self, logits, expert, dweights, dlogits, scoring="softmax", renormalise=True, scale=1.0, stream=None):
        """The gradient of the logits for ``dweights`` (tokens, k), with the
        choices ``expert`` of ``route`` held fixed."""
        dev = self.device
        T, E, ld, l_type = _matrix(logits, "logits", dev)
        rows, cols, ldd, d_type = _matrix(dlogits, "dlogits", dev)
        if (rows, cols, d_type) != (T, E, l_type):
            raise ValueError("dlogits must have the shape and type of logits")
        if expert.dim() != 2:
            raise ValueError("expert must be 2-D")
        k = expert.shape[1]
        flags = _route_flags(scoring, renormalise)
        e = _plain(expert, "expert", (T, k), "int64", dev)
        d = _plain(dweights, "dweights", (T, k), "float32", dev)
        with self._turn:
            rc = self._lib.gemm_route_grad(self.handle, T, E, k, logits.data_ptr(), ld, l_type, e, d, flags, scale,
                                           dlogits.data_ptr(), ldd, _raw_stream(stream, dev))
            if rc:
                self._check(rc)
        return dlogits

    def orthogonalise(self, G, out, steps=5, coefficients=(3.4445, -4.7750, 2.0315), eps=1e-7, stream=None):
        """The orthogonal factor of ``G``, or of every matrix of a batch, by
        Newton-Schulz steps, into ``out`` (which may be ``G``).

        X = G / (|G| + eps), then X <- a X + (b A + c A A) X with A = X X^T, or
        X^T X where that is smaller.  ``coefficients`` is (a, b, c), or one such
        triple a step.  float32 or bfloat16, out of G's type."""
        dev = self.device
        if G.dim() == 3:
            batch, rows, cols, ldg, sg, g_type = _matrices(G, "G", dev)
            got = _matrices(out, "out", dev)
        else:
            rows, cols, ldg, g_type = _matrix(G, "G", dev)
            batch, sg = 1, 0
            r, c, ld, o_type = _matrix(out, "out", dev)
            got = (1, r, c, ld, 0, o_type)
        if (got[0], got[1], got[2], got[5]) != (batch, rows, cols, g_type):
            raise ValueError("out must have the shape and type of G")
        table = _step_table(steps, coefficients)
        with self._turn:
            rc = self._lib.gemm_orthogonalise(self.handle, batch, rows, cols, G.data_ptr(), ldg, sg, out.data_ptr(),
                                              got[3], got[4], g_type, steps, table, eps, _raw_stream(stream, dev))
            if rc:
                self._check(rc)
        return out

    def mx4_quantise(self, src, out: Mx4, layout="col", stream=None):
        """Quantise ``src`` (float32 or bfloat16) along K into ``out``.

        ``layout="col"``: src is (rows, K), or (batch, rows, K); ``"row"``:
        (K, rows) or (batch, K, rows), turned on the way.  The matrices of a
        batch follow one another along out's rows."""
        lb = LAYOUTS.get(layout, layout)
        dev = self.device
        if src.dim() == 3:
            batch, d1, d2, ld, stride, s_type = _matrices(src, "src", dev)
        else:
            d1, d2, ld, s_type = _matrix(src, "src", dev)
            batch, stride = 1, 0
        rows, K = (d1, d2) if lb == GEMM_B_COL_MAJOR else (d2, d1)
        if out.rows != batch * rows or out.K != K:
            raise ValueError(f"out holds {out.rows} x {out.K}, src has {batch} x {rows} x {K}")
        with self._turn:
            rc = self._lib.gemm_mx4_quantise(self.handle, lb, batch, rows, K, src.data_ptr(), ld, stride, s_type,
                                             *out._args(dev), _raw_stream(stream, dev))
            if rc:
                self._check(rc)
        return out

    def mx4_dequantise(self, q: Mx4, out, stream=None):
        """The values ``q`` stands for, as float32 or bfloat16 (exact)."""
        dev = self.device
        rows, K, ld, o_type = _matrix(out, "out", dev)
        if rows != q.rows or K != q.K:
            raise ValueError(f"out has shape {tuple(out.shape)}, expected {(q.rows, q.K)}")
        with self._turn:
            rc = self._lib.gemm_mx4_dequantise(self.handle, rows, K, *q._args(dev), out.data_ptr(), ld, o_type,
                                               _raw_stream(stream, dev))
            if rc:
                self._check(rc)
        return out

    def run_mx4(self, A: Mx4, B: Mx4, C, stream=None):
        """C = A · B^T of two quantised matrices (M x K and N x K); C float32
        or bfloat16."""
        dev = self.device
        M, N, ldc, c_type = _matrix(C, "C", dev)
        if A.K != B.K or M != A.rows or N != B.rows:
            raise ValueError(f"shapes differ: A {A.rows} x {A.K}, B {B.rows} x {B.K}, C {tuple(C.shape)}")
        with self._turn:
            rc = self._lib.gemm_mx4_run(self.handle, M, N, A.K, *A._args(dev), *B._args(dev), C.data_ptr(), ldc,
                                        c_type, _raw_stream(stream, dev))
            if rc:
                self._check(rc)
        return C

    def run_mx4_grouped(self, A: Mx4, B: Mx4, offsets, C, stream=None):
        """``run_grouped`` of quantised operands: B holds the experts' N x K
        matrices one after another, N = C's columns."""
        dev = self.device
        M, N, ldc, c_type = _matrix(C, "C", dev)
        groups = offsets.shape[0] - 1
        if A.K != B.K or M != A.rows or B.rows != groups * N:
            raise ValueError(f"shapes differ: A {A.rows} x {A.K}, B {B.rows} x {B.K} for {groups} groups, "
                             f"C {tuple(C.shape)}")
        with self._turn:
            rc = self._lib.gemm_mx4_grouped_run(self.handle, groups, M, N, A.K, _offsets(offsets, groups, dev),
                                                *A._args(dev), *B._args(dev), C.data_ptr(), ldc, c_type,
                                                _raw_stream(stream, dev))
            if rc:
                self._check(rc)
        return C

    def i8_quantise(self, src, out: I8, layout="col", stream=None):
        """Quantise ``src`` (float32 or bfloat16) along K into ``out``, one scale a
        row; ``src`` and ``layout`` as in ``mx4_quantise``."""
        lb = LAYOUTS.get(layout, layout)
        dev = self.device
        if src.dim() == 3:
            batch, d1, d2, ld, stride, s_type = _matrices(src, "src", dev)
        else:
            d1, d2, ld, s_type = _matrix(src, "src", dev)
            batch, stride = 1, 0
        rows, K = (d1, d2) if lb == GEMM_B_COL_MAJOR else (d2, d1)
        if out.rows != batch * rows or out.K != K:
            raise ValueError(f"out holds {out.rows} x {out.K}, src has {batch} x {rows} x {K}")
        with self._turn:
            rc = self._lib.gemm_i8_quantise(self.handle, lb, batch, rows, K, src.data_ptr(), ld, stride, s_type,
                                            *out._args(dev), _raw_stream(stream, dev))
            if rc:
                self._check(rc)
        return out

    def i8_dequantise(self, q: I8, out, stream=None):
        """The values ``q`` stands for, code * scale, as float32 or bfloat16."""
        dev = self.device
        rows, K, ld, o_type = _matrix(out, "out", dev)
        if rows != q.rows or K != q.K:
            raise ValueError(f"out has shape {tuple(out.shape)}, expected {(q.rows, q.K)}")
        with self._turn:
            rc = self._lib.gemm_i8_dequantise(self.handle, rows, K, *q._args(dev), out.data_ptr(), ld, o_type,
                                              _raw_stream(stream, dev))
            if rc:
                self._check(rc)
        return out

    def run_i8(self, A: I8, B: I8, C, stream=None):
        """C = A · B^T of two 8-bit matrices (M x K and N x K), each sum of the
        codes' products times its row's and its column's scale; C float32 or
        bfloat16."""
        dev = self.device
        M, N, ldc, c_type = _matrix(C, "C", dev)
        if A.K != B.K or M != A.rows or N != B.rows:
            raise ValueError(f"shapes differ: A {A.rows} x {A.K}, B {B.rows} x {B.K}, C {tuple(C.shape)}")
        with self._turn:
            rc = self._lib.gemm_i8_run(self.handle, M, N, A.K, *A._args(dev), *B._args(dev), C.data_ptr(), ldc, c_type,
                                       _raw_stream(stream, dev))
            if rc:
                self._check(rc)
        return C

    def run_i8_grouped(self, A: I8, B: I8, offsets, C, stream=None):
        """``run_grouped`` of 8-bit operands: B holds the experts' N x K matrices
        one after another, N = C's columns."""
        dev = self.device
        M, N, ldc, c_type = _matrix(C, "C", dev)
        groups = offsets.shape[0] - 1
        if A.K != B.K or M != A.rows or B.rows != groups * N:
            raise ValueError(f"shapes differ: A {A.rows} x {A.K}, B {B.rows} x {B.K} for {groups} groups, "
                             f"C {tuple(C.shape)}")
        with self._turn:
            rc = self._lib.gemm_i8_grouped_run(self.handle, groups, M, N, A.K, _offsets(offsets, groups, dev),
                                               *A._args(dev), *B._args(dev), C.data_ptr(), ldc, c_type,
                                               _raw_stream(stream, dev))
            if rc:
                self._check(rc)
        return C

    def sync_status(self, stream=None):
        """Wait for ``stream`` and raise GemmError if an in-kernel wait expired or
        a call's group offsets were refused."""
        if stream is None:
            import torch
            stream = torch.cuda.current_stream()
        if hasattr(stream, "synchronize"):
            try:
                stream.synchronize()  # other threads' calls need not wait with this one
            except RuntimeError:
                pass  # the library reports it
        with self._turn:
            self._check(gemm_sync_status(self.handle, _stream_handle(stream)))

    @property
    def last_path(self) -> str:
        return gemm_last_path(self.handle)

    @property
    def launch_count(self) -> int:
        return gemm_launch_count(self.handle)


def matmul(A, B, layout_b="row", dtype="f32", out=None, stream=None, handle: Gemm | None = None):
    """Allocate C (float32, on A's device) if needed and return C = A·B."""
    import torch
    lb = LAYOUTS.get(layout_b, layout_b)
    M, N, _ = Gemm._dims(A, B, lb)
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=A.device)
    g = handle or default_handle(A.device.index or 0)
    return g.run(A, B, out, lb, dtype, stream)


def orthogonalise(G, steps=5, coefficients=(3.4445, -4.7750, 2.0315), eps=1e-7, out=None, stream=None,
                  handle: Gemm | None = None):
    """Allocate ``out`` (as G) if needed and return ``Gemm.orthogonalise``'s result."""
    import torch
    if G.device.type != "cuda":
        raise ValueError(f"G is on {G.device}: the products run on a CUDA device")
    if out is None:
        out = torch.empty(G.shape, dtype=G.dtype, device=G.device)
    g = handle or default_handle(G.device.index or 0)
    return g.orthogonalise(G, out, steps, coefficients, eps, stream)


_handles: dict[int, Gemm] = {}
_handles_lock = threading.Lock()


def default_handle(device: int | None = None) -> Gemm:
    """The handle of ``matmul`` and ``experts.grouped_matmul`` calls that name
    none, one per device (default: torch's current device).  All threads and
    streams share it; its ``sync_status`` reports what such calls found wrong on
    the GPU."""
    if device is None:
        import torch
        device = torch.cuda.current_device()
    with _handles_lock:
        h = _handles.get(device)
        if h is None:
            h = _handles[device] = Gemm(device)
    return h
