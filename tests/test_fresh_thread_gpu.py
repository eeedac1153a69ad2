"""Calls from host threads that have made no CUDA call of their own: their device
is reported as 0, but no context is current in them until the library makes it so."""
import threading

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


def in_a_thread(call):
    failures = []

    def work():
        try:
            call()
        except Exception as e:  # noqa: BLE001
            failures.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    assert not failures, failures


def test_products_from_a_fresh_thread(gm):
    """Everything a call needs is there already, the kernels' first use included."""
    A = torch.ones((96, 64), device="cuda").bfloat16()
    B = torch.ones((2, 64, 64), device="cuda").bfloat16()
    offsets = torch.tensor([0, 40, 96], device="cuda")
    C, W, D = (torch.zeros(s, device="cuda") for s in ((96, 64), (2, 64, 64), (96, 64)))
    with gm.Gemm(0) as h:
        h.run_grouped(A, B, offsets, C)
        h.run(A, B[0], D, "row", "bf16")
        h.sync_status()
        in_a_thread(lambda: h.run_grouped(A, B, offsets, C, stream=0))
        in_a_thread(lambda: h.run_grouped_wgrad(A, A, offsets, W, stream=0))
        in_a_thread(lambda: h.run(A, B[0], D, "row", "bf16", stream=0))
        torch.cuda.synchronize()
        h.sync_status()
    assert (C == 64).all() and (W[0] == 40).all() and (W[1] == 56).all() and (D == 64).all()
