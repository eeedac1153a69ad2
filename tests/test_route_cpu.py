"""The router's entry points without a GPU: declared functions are exported, the
header is plain C, arguments are checked on the host."""
import os
import re
import shutil
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gemm_route.h")
P = 0x10000  # a fake, aligned address: the checks never dereference


@pytest.fixture(scope="module")
def g():
    from dense_gemm_sm100_gb300 import build, gemm
    build.build()
    gemm.load_library()
    return gemm


def test_declared_functions_are_exported_and_bound(g):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(gemm_[a-z0-9_]+)\s*\(", text))
    assert len(names) == 4
    for n in names:
        assert hasattr(g.load_library(), n) and hasattr(g, n), n
    for n, value in re.findall(r"#define (GEMM_ROUTE_[A-Z_]+) (\d+)", text):
        assert getattr(g, n) == int(value)


def test_header_is_plain_c(tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("no gcc")
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    src = tmp_path / "use.c"
    src.write_text('#include "gemm_route.h"\nint main(void) { return GEMM_ROUTE_MAX_K > 0 ? 0 : 1; }\n')
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"),
                        "-isystem", os.path.join(cuda, "include"), "-c", str(src), "-o", str(tmp_path / "use.o")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


ROUTE = dict(tokens=8, experts=12, k=2, logits=P, ld=12, dtype=0, bias=P, groups=3, top_groups=2, flags=3, scale=1.0,
             weights=P, expert=P, order=P, offsets=P)


@pytest.mark.parametrize("change,code", [
    ({}, 0),
    ({"bias": 0}, 0),
    ({"dtype": 2}, 0),
    ({"dtype": 1}, -1),
    ({"flags": 4}, -1),
    ({"experts": 0}, -1),
    ({"experts": 1025, "ld": 1025, "groups": 1, "top_groups": 1}, -1),
    ({"experts": 1024, "ld": 1024, "groups": 32, "k": 31}, 0),
    ({"k": 0}, -1),
    ({"k": 8, "top_groups": 2}, 0),
    ({"k": 9, "top_groups": 2}, -1),         # two groups hold eight
    ({"k": 13, "top_groups": 3}, -1),
    ({"experts": 64, "ld": 64, "groups": 1, "top_groups": 1, "k": 32}, -1),
    ({"groups": 5}, -1),                     # not a divisor
    ({"groups": 0}, -1),
    ({"experts": 33 * 2, "ld": 66, "groups": 33}, -1),
    ({"top_groups": 0}, -1),
    ({"top_groups": 4}, -1),
    ({"tokens": -1}, -1),
    ({"tokens": (1 << 29) + 1}, -1),
    ({"tokens": 1 << 29}, 0),
    ({"tokens": 1 << 29, "ld": 1 << 16}, -1),
    ({"ld": 11}, -1),
    ({"ld": 1 << 37}, -1),
    ({"logits": 0}, -1),
    ({"weights": 0}, -1),
    ({"expert": 0}, -1),
    ({"order": 0}, -1),
    ({"offsets": 0}, -1),
    ({"logits": P + 2}, -2),
    ({"logits": P + 2, "dtype": 2}, 0),
    ({"logits": P + 1, "dtype": 2}, -2),
    ({"bias": P + 2}, -2),
    ({"weights": P + 2}, -2),
    ({"expert": P + 4}, -2),
    ({"order": P + 4}, -2),
    ({"offsets": P + 4}, -2),
    ({"tokens": 0, "logits": 0, "weights": 0, "expert": 0, "order": 0}, 0),
    ({"tokens": 0, "offsets": 0}, -1),       # zeros are written
])
def test_route_arguments(g, change, code):
    assert g.gemm_route_validate(*{**ROUTE, **change}.values()) == code


GRAD = dict(tokens=8, experts=12, k=2, logits=P, ld=12, dtype=0, expert=P, dweights=P, flags=3, scale=1.0, dlogits=P,
            ldd=12)


@pytest.mark.parametrize("change,code", [
    ({}, 0),
    ({"dtype": 3}, -1),
    ({"flags": -1}, -1),
    ({"k": 13}, -1),
    ({"ld": 11}, -1),
    ({"ldd": 11}, -1),
    ({"ldd": 1 << 37}, -1),
    ({"tokens": 1 << 29, "ldd": 1 << 16}, -1),
    ({"expert": 0}, -1),
    ({"dweights": 0}, -1),
    ({"dlogits": 0}, -1),
    ({"expert": P + 4}, -2),
    ({"dweights": P + 1}, -2),
    ({"dlogits": P + 2}, -2),
    ({"dlogits": P + 2, "dtype": 2}, 0),
    ({"tokens": 0, "logits": 0, "expert": 0, "dweights": 0, "dlogits": 0}, 0),
])
def test_grad_arguments(g, change, code):
    assert g.gemm_route_grad_validate(*{**GRAD, **change}.values()) == code


def test_calls_without_a_handle_are_refused(g):
    assert g.gemm_route(None, *ROUTE.values(), None) == g.GEMM_ERR_INVALID
    assert g.gemm_route_grad(None, *GRAD.values(), None) == g.GEMM_ERR_INVALID


def test_cpu_tensors_are_refused(g):
    from dense_gemm_sm100_gb300.experts import route
    with pytest.raises(ValueError, match="CUDA device"):
        route(torch.zeros(2, 4), 2)


def test_binding_checks_without_a_device(g):
    """The checks of scoring and shapes come before any call into the library."""
    with pytest.raises(ValueError, match="scoring"):
        g._route_flags("relu", True)
    assert g._route_flags("sigmoid", False) == g.GEMM_ROUTE_SIGMOID
    out = g.routing_empty(3, 5, 2, device="cpu")
    assert out.weights.shape == (3, 2) and out.order.shape == (6,) and out.offsets.shape == (6,)
    assert out.expert.dtype == torch.int64


def test_weights_of_follows_the_definition(g):
    """The torch form behind gradients of gradients, on the CPU."""
    from dense_gemm_sm100_gb300.experts import _weights_of
    gen = torch.Generator().manual_seed(2)
    x = torch.randn((6, 7), generator=gen)
    x[4] = float("-inf")
    expert = torch.tensor([[0, 3], [6, 2], [1, -1], [5, 4], [-1, -1], [2, 0]])
    for scoring in ("softmax", "sigmoid"):
        for renormalise in (True, False):
            w = _weights_of(x, expert, scoring, renormalise, 2.0)
            for t in range(6):
                p = torch.softmax(x[t].double(), 0) if scoring == "softmax" else torch.sigmoid(x[t].double())
                s = torch.tensor([p[e] if e >= 0 else 0.0 for e in expert[t].tolist()], dtype=torch.float64)
                ref = 2 * (s / (s.sum() + 1e-20) if renormalise else s)
                assert (w[t].double() - ref).abs().max() <= 2.0 ** -20
            leaf = x.clone().requires_grad_()
            grad, = torch.autograd.grad(_weights_of(leaf, expert, scoring, renormalise, 1.0).square().sum(), leaf)
            assert torch.isfinite(grad).all() and (grad[4] == 0).all()
