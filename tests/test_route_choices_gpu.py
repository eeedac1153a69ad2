"""The router's choices where values are close, equal, saturated or infinite,
compared in every combination with the definition in 64 bits.

Weights: (2 d + E / 32 + 18) u of themselves, u = 2^-24, d the row's span of finite
logits (exp within 2 ulp of an argument off by d u, twice, a sum of E terms, a
division), plus 2^-126 where a score leaves FP32's normal numbers.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def gm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dense_gemm_sm100_gb300 import build, gemm
    build.build()
    return gemm


@pytest.fixture()
def h(gm):
    with gm.Gemm(0) as handle:
        yield handle


def definition(logits, k, scoring, bias=None, groups=1, top_groups=1, renormalise=True):
    """(weights, expert) in 64 bits, row by row; a bias of minus infinity excludes."""
    T, E = logits.shape
    weights, expert = torch.zeros((T, k), dtype=torch.float64), torch.full((T, k), -1)
    b = torch.zeros(E, dtype=torch.float64) if bias is None else bias.double()
    for t in range(T):
        x = logits[t].double()
        if torch.isnan(x).any() or (scoring == "softmax" and (x == math.inf).any()):
            weights[t] = math.nan
            continue
        if (x == -math.inf).all():
            continue
        s = 1 / (1 + torch.exp(-x)) if scoring == "sigmoid" else torch.softmax(x, 0)
        value = s + b
        live = [e for e in range(E) if x[e] > -math.inf and b[e] > -math.inf]
        if groups > 1:
            n, best = E // groups, []
            for g in range(groups):
                inside = sorted((float(value[e]) for e in live if e // n == g), reverse=True)
                if inside:
                    best.append((-sum(inside[:2]), g))
            kept = {g for _, g in sorted(best)[:top_groups]}
            live = [e for e in live if e // n in kept]
        rank = x if bias is None else value
        first = sorted(live, key=lambda e: (-float(rank[e]), e))[:k]
        if not first:
            continue
        if not renormalise:
            w = s[first]
        elif scoring == "sigmoid":
            w = s[first] / (s[first].sum() + 1e-20)
        else:
            w = torch.softmax(x[first], 0)
        weights[t, :len(first)] = w
        expert[t, :len(first)] = torch.tensor(first)
    return weights, expert


def routed(gm, h, x, k, *args, **kw):
    r = gm.routing_empty(x.shape[0], x.shape[1], k)
    r.weights.fill_(-7)
    for t in (r.expert, r.order, r.offsets):
        t.fill_(-9)
    bias = kw.pop("bias", None)
    h.route(x.cuda(), r, *args, bias=None if bias is None else bias.cuda(), **kw)
    h.sync_status()
    flat = r.expert.flatten().cpu()
    want = torch.sort(flat, stable=True)
    assert torch.equal(r.order.cpu(), want.indices)
    assert torch.equal(r.offsets.cpu(), torch.searchsorted(want.values, torch.arange(x.shape[1] + 1)))
    return r


def weights_near(r, w, x):
    got = r.weights.cpu().double()
    assert torch.equal(torch.isnan(got), torch.isnan(w))
    for t in range(x.shape[0]):
        if torch.isnan(w[t]).any():
            continue
        fine = x[t].double()[torch.isfinite(x[t])]
        d = float(fine.max() - fine.min()) if fine.numel() else 0.0
        # a span past 200 leaves scores of 0 and 1 in FP32, or as near as 2^-126
        tol = (2 * min(d, 200.0) + x.shape[1] / 32 + 18) * U * w[t] + 2.0 ** -126
        assert ((got[t] - w[t]).abs() <= tol).all(), (t, got[t], w[t])


@pytest.mark.parametrize("k", [1, 4, 8, 9])
@pytest.mark.parametrize("renormalise", [True, False])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("kind", ["none", "finite", "excluding", "forcing", "both"])
def test_odd_values(gm, h, kind, scoring, renormalise, k):
    x = torch.randn((12, 40), generator=torch.Generator().manual_seed(1))
    x[0, 3] = math.nan
    x[1, 4] = math.inf
    x[2] = -math.inf
    x[3] = x[3] * 1e30
    x[4, ::2] = -3e38
    x[5] = -500.0  # sigmoid scores below the smallest float
    x[6, 5:] = -math.inf
    bias = None if kind == "none" else torch.zeros(40)
    if kind in ("finite", "both"):
        bias[20:30] = 0.25
    if kind in ("excluding", "both"):
        bias[7] = -math.inf
    if kind in ("forcing", "both"):
        bias[11] = math.inf
    r = routed(gm, h, x, k, scoring, bias=bias, renormalise=renormalise)
    w, e = definition(x, k, scoring, bias, renormalise=renormalise)
    assert torch.equal(r.expert.cpu(), e)
    weights_near(r, w, x)


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [24, 96, 250, 700])
def test_groups_of_neighbouring_logits(gm, h, E, scoring, sign):
    """FP32 logits one unit in the last place apart, each twice: sums of a group's two
    best that differ by 1e-8, or not at all."""
    gen = torch.Generator().manual_seed(2)
    steps = torch.stack([torch.randperm(E, generator=gen) for _ in range(70)])
    x = sign * (1.0 + (steps // 2).float() * 2.0 ** -23)
    for k, groups, top in ((3, 2, 1), (2, 2, 1), (8, 2, 1)):
        r = routed(gm, h, x, k, scoring, groups=groups, top_groups=top)
        _, e = definition(x, k, scoring, None, groups, top)
        assert torch.equal(r.expert.cpu(), e)


@pytest.mark.parametrize("draw", range(6))
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_close_sums_of_different_rows(gm, h, scoring, draw):
    """A bias that all but cancels the differences of the scores of one row; the rows
    are that row moved by up to 1 (softmax: the scores stay, up to the rounding of the
    logits, 1e-7) or by 1e-6 (sigmoid)."""
    gen = torch.Generator().manual_seed(10 + draw)
    E, T = (48, 160, 400)[draw % 3], 64
    x = torch.randn((1, E), generator=gen)
    s = torch.softmax(x[0].double(), 0) if scoring == "softmax" else torch.sigmoid(x[0].double())
    step = torch.randperm(E, generator=gen).double() * (4e-8 if scoring == "sigmoid" else 4e-9)
    bias = (0.9 - s + step).float()
    shift = torch.randn((T, 1), generator=gen)
    x = x + (shift if scoring == "softmax" else 1e-6 * shift)
    assert len(torch.unique(x, dim=0)) > T // 2
    for groups, top, k in ((1, 1, 8), (1, 1, 12), (4, 2, 8), (8, 3, 5)):
        r = routed(gm, h, x, k, scoring, bias=bias, groups=groups, top_groups=top)
        w, e = definition(x, k, scoring, bias, groups, top)
        assert torch.equal(r.expert.cpu(), e)
        weights_near(r, w, x)


@pytest.mark.parametrize("low", [-3.4028234663852886e38, -1e38, -1e9])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,top,k", [(8, 4, 4, 8), (8, 4, 2, 4), (64, 8, 6, 8), (96, 8, 8, 31), (640, 8, 3, 9),
                                           (12, 1, 1, 8)])
def test_biases_of_the_lowest_value(gm, h, E, groups, top, k, scoring, low):
    """A finite bias, the type's lowest one too, ranks last and excludes nothing: sums
    of a group's two best may leave FP32."""
    gen = torch.Generator().manual_seed(3)
    x = torch.randn((40, E), generator=gen)
    x[20:, ::3] = -math.inf
    for masked in (torch.arange(E) % (E // groups) < E, torch.arange(E) >= E // 2,
                   torch.rand(E, generator=gen) < 0.8):
        bias = torch.where(masked, low, 0.1 * torch.randn(E, generator=gen))
        bias[E // 3] = low / 2
        r = routed(gm, h, x, k, scoring, bias=bias, groups=groups, top_groups=top)
        w, e = definition(x, k, scoring, bias, groups, top)
        assert torch.equal(r.expert.cpu(), e)
        weights_near(r, w, x)
