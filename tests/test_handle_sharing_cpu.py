"""Handles that several host threads share, without a GPU: the library's calls
are replaced by ones that notice company."""
import threading
import time

import pytest
import torch

from dense_gemm_sm100_gb300 import gemm as g


class Busy:
    """Stands in for the C calls: counts calls that overlap."""

    def __init__(self):
        self.inside = self.overlaps = self.calls = 0

    def __call__(self, *args):
        self.inside += 1
        self.overlaps += self.inside > 1
        time.sleep(0.002)
        self.calls += 1
        self.inside -= 1
        return 0

    def __getattr__(self, name):  # any function of the library
        return self


class DeviceTensor:
    """A contiguous tensor's fields, on a device that is not there."""

    is_cuda = True

    def __init__(self, dtype, *shape):
        self.shape, self.dtype = shape, dtype
        self._stride = torch.empty(shape, device="meta").stride()

    def get_device(self):
        return 0

    def stride(self, d=None):
        return self._stride if d is None else self._stride[d]

    def dim(self):
        return len(self.shape)

    def data_ptr(self):
        return 1 << 20


@pytest.fixture()
def shared(monkeypatch):
    busy = Busy()
    monkeypatch.setattr(g, "gemm_create", lambda device: 1)
    monkeypatch.setattr(g, "gemm_destroy", lambda handle: 0)
    monkeypatch.setattr(g, "load_library", lambda: busy)
    for name in ("gemm_run", "gemm_run_host", "gemm_sync_status", "gemm_set_option"):
        monkeypatch.setattr(g, name, busy)
    handle = g.Gemm(0)
    yield handle, busy
    handle.handle = None  # not one that the library could destroy


def in_threads(n, f):
    threads = [threading.Thread(target=f) for _ in range(n)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()


def test_calls_of_several_threads_take_turns(shared):
    h, busy = shared
    bf16, f32 = torch.bfloat16, torch.float32
    a, w, c = DeviceTensor(bf16, 8, 32), DeviceTensor(bf16, 2, 32, 16), DeviceTensor(f32, 8, 16)
    x, dw, o = DeviceTensor(bf16, 8, 16), DeviceTensor(f32, 2, 32, 16), DeviceTensor(torch.int64, 3)
    b, q = DeviceTensor(f32, 32, 16), g.Mx4(torch.zeros(8, 16, dtype=torch.uint8), torch.zeros(8, 16, dtype=torch.uint8), 32)
    q._device = 0
    a32 = DeviceTensor(f32, 8, 32)

    def work():
        h.run(a32, b, c, "row", "f32", stream=0)
        h.run_host(a32, b, c, "row", "f32", stream=0)
        h.run_grouped(a, w, o, c, "row", "bf16", stream=0)
        h.run_grouped_wgrad(a, x, o, dw, "bf16", stream=0)
        h.mx4_quantise(a, q, stream=0)
        h.mx4_dequantise(q, a, stream=0)
        h.run_mx4(q, q, DeviceTensor(f32, 8, 8), stream=0)
        h.run_mx4_grouped(q, q, o, DeviceTensor(f32, 8, 4), stream=0)
        h.set_option(1, 0)
        h.sync_status(0)

    in_threads(4, work)
    assert busy.calls == 40 and busy.overlaps == 0


def test_threads_get_one_default_handle(monkeypatch):
    made = []

    class Slow:
        def __init__(self, device):
            time.sleep(0.01)
            made.append(device)

    monkeypatch.setattr(g, "Gemm", Slow)
    monkeypatch.setattr(g, "_handles", {})
    got = []
    in_threads(4, lambda: got.append(g.default_handle(0)))
    assert made == [0] and len(set(map(id, got))) == 1
    assert g.default_handle(0) is got[0] and g.default_handle(1) is not got[0]


def test_dense_operands_whose_rows_overlap_are_refused(shared):
    """An expanded operand would be read at the pitch of its columns, past the
    end of its storage."""
    h, busy = shared
    a, b, c = torch.zeros(4, 8), torch.zeros(8, 4), torch.zeros(4, 4)
    row = torch.zeros(1, 8)
    for args in ((row.expand(4, 8), b, c), (a, torch.zeros(1, 4).expand(8, 4), c), (a, b, torch.zeros(1, 4).expand(4, 4)),
                 (torch.zeros(32).as_strided((4, 8), (4, 1)), b, c)):
        for run in (h.run, h.run_host):
            with pytest.raises(ValueError):
                run(*args, stream=0)
    assert busy.calls == 0
    h.run(row.expand(1, 8), b, c[:1], stream=0)
    h.run(torch.zeros(4, 16)[:, :8], b, c, stream=0)
    assert busy.calls == 2
