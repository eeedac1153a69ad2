"""The expert router on the GPU against its definition, row by row in 64 bits.

Tolerances (u = 2^-24).  A score in FP32: exp within 2 ulp (4 u) of an argument
that is itself off by |x - max| u, twice for a quotient of two; a sum of E terms
in rows of 32 lanes adds (E / 32 + 5) u, the division and the scale 3 u.  So a
weight is off by (2 d + E / 32 + 18) u of itself, d = the largest |x - max| of a
chosen logit (rounded up to the row's span).  A gradient is a sum of at most
k + 1 products of such weights: (4 (2 d + E / 32 + 18) + k + 8) u of the sum of
the products' sizes, and half a step of its type.
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


def scores_of(x, scoring):
    if scoring == "sigmoid":
        return torch.sigmoid(x.double())
    return torch.softmax(x.double(), 0)


def definition(logits, k, scoring="softmax", bias=None, groups=1, top_groups=1, renormalise=True, scale=1.0):
    """(weights, expert) in 64 bits, row by row."""
    T, E = logits.shape
    weights, expert = torch.zeros((T, k), dtype=torch.float64), torch.full((T, k), -1)
    for t in range(T):
        x = logits[t].double().cpu()
        if torch.isnan(x).any() or (scoring == "softmax" and (x == math.inf).any()):
            weights[t] = math.nan
            continue
        live = [e for e in range(E) if x[e] > -math.inf]
        if not live:
            continue
        s = scores_of(x, scoring)
        value = s + (bias.double().cpu() if bias is not None else 0.0)
        if groups > 1:
            n = E // groups
            best = []
            for g in range(groups):
                inside = sorted((float(value[e]) for e in live if e // n == g), reverse=True)
                if inside:
                    best.append((-sum(inside[:2]), g))
            kept = {g for _, g in sorted(best)[:top_groups]}
            live = [e for e in live if e // n in kept]
        rank = value if bias is not None else x
        first = sorted(live, key=lambda e: (-float(rank[e]), e))[:k]
        chosen = s[first]
        if renormalise:
            chosen = chosen / (chosen.sum() + (1e-20 if scoring == "sigmoid" else 0.0))
        weights[t, :len(first)] = scale * chosen
        expert[t, :len(first)] = torch.tensor(first)
    return weights, expert


def gradient(logits, expert, dweights, scoring, renormalise, scale):
    """(dlogits, sum of the sizes of its terms) by the formula, row by row."""
    T, E = logits.shape
    d, size = torch.zeros((T, E), dtype=torch.float64), torch.zeros((T, E), dtype=torch.float64)
    for t in range(T):
        at = [(i, e) for i, e in enumerate(expert[t].tolist()) if e >= 0]
        if not at:
            continue
        x = logits[t].double()
        s = scores_of(x, scoring)
        jac = torch.zeros((len(at), E), dtype=torch.float64)  # of the chosen scores
        for n, (_, e) in enumerate(at):
            if scoring == "sigmoid":
                jac[n, e] = s[e] * torch.sigmoid(-x[e])
            else:
                jac[n] = -s[e] * s
                jac[n, e] += s[e]
        p = torch.stack([s[e] for _, e in at])
        g = scale * torch.stack([dweights[t, i].double() for i, _ in at])
        if renormalise:
            total = p.sum() + (1e-20 if scoring == "sigmoid" else 0.0)
            outer = torch.diag(1 / total.expand(len(at))) - (p / total ** 2)[:, None]
            jac = outer @ jac
            if scoring == "softmax":  # sizes: w (|g| + sum w |g|); the rest cancels to zero
                w = p / total
                for n, (_, e) in enumerate(at):
                    size[t, e] += w[n] * (g[n].abs() + (w * g.abs()).sum())
            else:
                w = p / total
                for n, (_, e) in enumerate(at):
                    size[t, e] += (g[n].abs() + (w * g.abs()).sum()) / total * s[e] * torch.sigmoid(-x[e])
        else:
            if scoring == "softmax":
                size[t] = s * (p * g.abs()).sum()
            for n, (_, e) in enumerate(at):
                size[t, e] += p[n] * g[n].abs()
        d[t] = g @ jac
        if renormalise and scoring == "softmax":
            out = torch.ones(E, dtype=torch.bool)
            out[[e for _, e in at]] = False
            d[t, out] = 0.0  # exactly: the denominators cancel
    return d, size


def weight_tolerance(logits, E):
    x = logits.double().cpu()
    x = x[torch.isfinite(x)]
    span = float(x.max() - x.min()) if x.numel() else 0.0
    return (2 * span + E / 32 + 18) * U


def check_sorted(r, E):
    flat = r.expert.flatten().cpu()
    order, offsets = r.order.cpu(), r.offsets.cpu()
    want = torch.sort(flat, stable=True)
    assert torch.equal(order, want.indices)
    assert torch.equal(offsets, torch.searchsorted(want.values, torch.arange(E + 1)))


def fresh(gm, T, E, k):
    r = gm.routing_empty(T, E, k)
    r.weights.fill_(-7)
    for t in (r.expert, r.order, r.offsets):
        t.fill_(-9)
    return r


def draw_logits(T, E, dtype, seed, masked=0.1):
    gen = torch.Generator().manual_seed(seed)
    x = 2 * torch.randn((T, E), generator=gen)
    x[torch.rand((T, E), generator=gen) < masked] = -math.inf
    if T > 2:
        x[T // 2] = -math.inf  # a row of padding
        x[1, 1:] = -math.inf   # one choice
    return x.to(dtype)


SHAPES = [(1, 1, 1), (1, 8, 2), (2, 31, 3), (7, 33, 8), (64, 60, 4), (65, 64, 8), (33, 128, 31), (130, 256, 8),
          (200, 300, 5), (70, 520, 9), (40, 1024, 31)]


@pytest.mark.parametrize("renormalise", [True, False])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", SHAPES)
def test_route_matches_the_definition(gm, h, T, E, k, dtype, scoring, renormalise):
    x = draw_logits(T, E, dtype, 3)
    r = fresh(gm, T, E, k)
    h.route(x.cuda(), r, scoring, renormalise=renormalise, scale=1.5)
    h.sync_status()
    w, e = definition(x, k, scoring, renormalise=renormalise, scale=1.5)
    assert torch.equal(r.expert.cpu(), e)
    assert ((r.weights.cpu().double() - w).abs() <= weight_tolerance(x, E) * w).all()
    check_sorted(r, E)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,groups,top", [(3, 4, 2, 2, 1), (40, 60, 4, 3, 2), (90, 64, 8, 8, 4), (70, 256, 8, 8, 4),
                                             (50, 96, 5, 32, 7), (33, 32, 3, 32, 32), (20, 1024, 31, 16, 16),
                                             (5, 7, 3, 1, 1)])
@pytest.mark.parametrize("biased", [True, False])
def test_bias_and_groups(gm, h, T, E, k, groups, top, scoring, biased):
    x = draw_logits(T, E, torch.float32, 5)
    gen = torch.Generator().manual_seed(6)
    bias = 0.2 * torch.randn(E, generator=gen) if biased else None
    r = fresh(gm, T, E, k)
    h.route(x.cuda(), r, scoring, bias.cuda() if biased else None, groups, top)
    h.sync_status()
    w, e = definition(x, k, scoring, bias, groups, top)
    assert torch.equal(r.expert.cpu(), e)
    assert ((r.weights.cpu().double() - w).abs() <= weight_tolerance(x, E) * w).all()
    check_sorted(r, E)


def test_equal_values_rank_by_index(gm, h):
    """Few different logits, zeros of both signs among them: ties everywhere."""
    gen = torch.Generator().manual_seed(7)
    x = torch.randint(-1, 2, (150, 96), generator=gen).float()
    x[torch.rand(x.shape, generator=gen) < 0.3] = -0.0
    for bias, groups, top in ((None, 1, 1), (torch.zeros(96), 1, 1), (None, 8, 3), (torch.full((96,), 0.25), 8, 3)):
        for scoring in ("softmax", "sigmoid"):
            r = fresh(gm, 150, 96, 8)
            h.route(x.cuda(), r, scoring, None if bias is None else bias.cuda(), groups, top)
            _, e = definition(x, 8, scoring, bias, groups, top)
            assert torch.equal(r.expert.cpu(), e)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_close_sums_are_decided_in_64_bits(gm, h, scoring):
    """Biases that all but cancel the scores' differences: the sums differ by
    1e-9 to 1e-7, below what FP32 scores can tell, and the exact order counts."""
    gen = torch.Generator().manual_seed(8)
    E, T = 48, 64
    x = torch.randn((1, E), generator=gen).expand(T, E).contiguous()
    s = scores_of(x[0], scoring)
    step = torch.randperm(E, generator=gen).double() * 4e-8
    bias = (0.9 - s + step).float()  # its own rounding (3e-8) makes the order the exact sums'
    shift = 1e-6 * torch.randn((T, 1), generator=gen) if scoring == "sigmoid" else torch.zeros((T, 1))
    x = x + shift
    for groups, top, k in ((1, 1, 12), (6, 3, 8)):
        r = fresh(gm, T, E, k)
        h.route(x.cuda(), r, scoring, bias.cuda(), groups, top)
        _, e = definition(x, k, scoring, bias, groups, top)
        assert torch.equal(r.expert.cpu(), e)


@pytest.mark.parametrize("biased", [True, False])
@pytest.mark.parametrize("E,groups", [(16, 4), (256, 8), (640, 8)])
def test_scores_near_the_smallest_number(gm, h, E, groups, biased):
    """Sigmoids of 1e-39 to 1e-36, some of which FP32 has only as zero."""
    gen = torch.Generator().manual_seed(12)
    x = -90 + 6 * torch.rand((100, E), generator=gen)
    bias = torch.zeros(E) if biased else None
    r = fresh(gm, 100, E, 4)
    h.route(x.cuda(), r, "sigmoid", bias.cuda() if biased else None, groups, 2)
    _, e = definition(x, 4, "sigmoid", bias, groups, 2)
    assert torch.equal(r.expert.cpu(), e)


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_neighbouring_logits_keep_their_order(gm, h, sign):
    """FP32 logits one unit in the last place apart, and equal ones."""
    gen = torch.Generator().manual_seed(23)
    for E in (24, 96, 250, 700):
        steps = torch.stack([torch.randperm(E, generator=gen) for _ in range(70)])
        x = sign * (1.0 + (steps // 2).float() * 2.0 ** -23)
        for k, groups, top in ((8, 1, 1), (3, 2, 1), (8, 2, 2)):
            r = fresh(gm, 70, E, k)
            h.route(x.cuda(), r, "sigmoid", None, groups, top)
            if groups == 1 or top == groups:
                assert torch.equal(r.expert.cpu(), definition(x, k, "sigmoid")[1])
            check_sorted(r, E)


def test_odd_values(gm, h):
    """NaN, infinities, far logits, biases that exclude or force an expert."""
    x = torch.randn((12, 40), generator=torch.Generator().manual_seed(9))
    x[0, 3] = math.nan
    x[1, 4] = math.inf
    x[2] = -math.inf
    x[3] = x[3] * 1e30
    x[4, ::2] = -3e38
    x[5] = -500.0  # sigmoid scores below the smallest float
    bias = torch.zeros(40)
    bias[7], bias[11] = -math.inf, math.inf
    for scoring in ("softmax", "sigmoid"):
        for b in (None, bias):
            r = fresh(gm, 12, 40, 4)
            h.route(x.cuda(), r, scoring, None if b is None else b.cuda())
            if b is None:
                w, e = definition(x, 4, scoring)
            else:
                masked = x.clone()
                masked[:, 7] = torch.where(torch.isnan(x[:, 7]), x[:, 7], -math.inf)
                w, e = definition(masked, 4, scoring, torch.where(b == -math.inf, 0.0, b))
            if scoring == "softmax" or b is None:
                assert torch.equal(r.expert.cpu(), e)
            got = r.weights.cpu().double()
            assert torch.equal(torch.isnan(got), torch.isnan(w))
            assert (r.expert[0] == -1).all() and (r.expert[2] == -1).all() and (r.weights[2] == 0).all()
            if b is not None:
                assert not (r.expert == 7).any() and (r.expert[6:, 0] == 11).all()
            fine = [6, 7, 8, 9, 10, 11]
            if scoring == "softmax" and b is not None:  # the sum is over every logit; renormalised, it cancels
                w, _ = definition(x, 4, scoring, torch.where(b == -math.inf, -1e9, b))
            assert ((got[fine] - w[fine]).abs() <= weight_tolerance(x[6:], 40) * w[fine]).all()
            check_sorted(r, 40)


@pytest.mark.parametrize("T", [0, 1, 63, 64, 65, 4000, 20011])
def test_many_tokens_are_sorted(gm, h, T):
    x = draw_logits(T, 64, torch.bfloat16, 10)
    r = fresh(gm, T, 64, 6)
    h.route(x.cuda(), r)
    h.sync_status()
    check_sorted(r, 64)
    if T:
        # choices by an independent stable sort of the logits
        value, index = torch.sort(x.float(), dim=1, descending=True, stable=True)
        want = torch.where(value[:, :6] > -math.inf, index[:, :6], -1)
        assert torch.equal(r.expert.cpu(), want)
    else:
        assert (r.offsets == 0).all()


def test_all_tokens_to_one_expert(gm, h):
    x = torch.zeros((3000, 16), device="cuda")
    x[:, 5] = 1
    r = fresh(gm, 3000, 16, 1)
    h.route(x, r)
    assert torch.equal(r.order, torch.arange(3000, device="cuda"))
    assert r.offsets.tolist() == [0] * 6 + [3000] * 11 and (r.weights == 1).all()


def test_strided_logits(gm, h):
    wide = torch.randn((90, 70), generator=torch.Generator().manual_seed(11)).cuda()
    x = wide[:, 3:53]
    a, b = fresh(gm, 90, 50, 4), fresh(gm, 90, 50, 4)
    h.route(x, a)
    h.route(x.contiguous(), b)
    for u, v in zip(a, b):
        assert torch.equal(u, v)
    d = torch.full((90, 70), 5.0, device="cuda")
    dw = torch.randn((90, 4), device="cuda")
    ref = torch.empty((90, 50), device="cuda")
    h.route_grad(x, a.expert, dw, d[:, 3:53], renormalise=False)
    h.route_grad(x.contiguous(), a.expert, dw, ref, renormalise=False)
    assert torch.equal(d[:, 3:53], ref) and (d[:, :3] == 5).all() and (d[:, 53:] == 5).all()


@pytest.mark.parametrize("renormalise", [True, False])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 8, 2), (40, 60, 4), (33, 128, 8), (30, 300, 5), (9, 1023, 31)])
def test_gradient_matches_the_formula(gm, h, T, E, k, dtype, scoring, renormalise):
    x = draw_logits(T, E, dtype, 12)
    r = fresh(gm, T, E, k)
    h.route(x.cuda(), r, scoring, renormalise=renormalise, scale=1.5)
    dw = torch.randn((T, k), generator=torch.Generator().manual_seed(13))
    got = torch.full((T, E), math.nan, dtype=dtype, device="cuda")
    h.route_grad(x.cuda(), r.expert, dw.cuda(), got, scoring, renormalise, 1.5)
    h.sync_status()
    d, size = gradient(x, r.expert.cpu(), dw, scoring, renormalise, 1.5)
    tol = (4 * weight_tolerance(x, E) + (k + 8) * U) * size + torch.finfo(dtype).eps / 2 * d.abs() + 1e-40
    assert ((got.cpu().double() - d).abs() <= tol).all()


@pytest.mark.parametrize("renormalise", [True, False])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_gradient_matches_differences(gm, scoring, renormalise):
    """Through autograd, against central differences of the 64-bit definition
    (step 1e-4: its error is 1e-8 of third derivatives below 1) and FP32 weights."""
    from dense_gemm_sm100_gb300.experts import route
    x = draw_logits(12, 20, torch.float32, 14)
    gen = torch.Generator().manual_seed(15)
    dw = torch.randn((12, 3), generator=gen)
    leaf = x.cuda().requires_grad_()
    r = route(leaf, 3, scoring, renormalise=renormalise, scale=2.0)
    (r.weights * dw.cuda()).sum().backward()
    expert = r.expert.cpu()

    def value(logits, t):
        s = scores_of(logits, scoring)
        at = [(i, e) for i, e in enumerate(expert[t].tolist()) if e >= 0]
        p = torch.stack([s[e] for _, e in at])
        if renormalise:
            p = p / (p.sum() + (1e-20 if scoring == "sigmoid" else 0.0))
        return 2.0 * sum(p[n] * dw[t, i].double() for n, (i, _) in enumerate(at))

    for t in range(12):
        if (expert[t] < 0).all():
            assert (leaf.grad[t] == 0).all()
            continue
        for e in range(0, 20, 3):
            if x[t, e] == -math.inf:
                assert leaf.grad[t, e] == 0
                continue
            lo, hi = x[t].double(), x[t].double()
            lo[e] -= 1e-4
            hi[e] += 1e-4
            diff = (value(hi, t) - value(lo, t)) / 2e-4
            assert abs(float(diff) - float(leaf.grad[t, e])) <= 3e-6


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [True, False])
def test_second_order_gradients(gm, scoring, renormalise):
    """create_graph gives the same first gradient, and a second one that matches
    torch's own of the weights in 64 bits."""
    from dense_gemm_sm100_gb300.experts import _weights_of, route
    x = torch.randn((10, 24), generator=torch.Generator().manual_seed(16)).cuda()
    dw = torch.randn((10, 4), generator=torch.Generator().manual_seed(17)).cuda()
    a = x.clone().requires_grad_()
    r = route(a, 4, scoring, renormalise=renormalise)
    first, = torch.autograd.grad(r.weights, a, dw, create_graph=True)
    second, = torch.autograd.grad(first.square().sum(), a)
    b = x.clone().requires_grad_()
    plain, = torch.autograd.grad(route(b, 4, scoring, renormalise=renormalise).weights, b, dw)
    assert (first - plain).abs().max() <= 64 * U * 4
    c = x.double().requires_grad_()
    s = torch.sigmoid(c) if scoring == "sigmoid" else torch.softmax(c, -1)
    w = torch.gather(s, 1, r.expert)
    if renormalise:
        w = w / w.sum(-1, keepdim=True)
    g, = torch.autograd.grad(w, c, dw.double(), create_graph=True)
    want, = torch.autograd.grad(g.square().sum(), c)
    assert (second - want).abs().max() <= 1e-5 * want.abs().max()


def test_foreign_choices_do_no_harm(gm, h):
    """Indices outside the experts count for nothing, one that comes twice counts twice."""
    x = torch.randn((4, 10), generator=torch.Generator().manual_seed(18))
    expert = torch.tensor([[3, 3], [-5, 2], [10, 1 << 40], [9, 0]])
    dw = torch.ones((4, 2))
    got = torch.empty((4, 10), device="cuda")
    h.route_grad(x.cuda(), expert.cuda(), dw.cuda(), got, "sigmoid", renormalise=False)
    s = torch.sigmoid(x.double())
    d = s * (1 - s)
    want = torch.zeros((4, 10), dtype=torch.float64)
    want[0, 3] = 2 * d[0, 3]
    want[1, 2] = d[1, 2]
    want[3, 9], want[3, 0] = d[3, 9], d[3, 0]
    assert (got.cpu().double() - want).abs().max() <= 32 * U


def test_streams_and_captured_graphs(gm, h):
    """A captured call replays on new logits; another stream's call on the same
    handle takes its turn with the workspace."""
    gen = torch.Generator().manual_seed(19)
    xs = [torch.randn((500, 64), generator=gen).cuda() for _ in range(3)]
    want = []
    for x in xs:
        r = fresh(gm, 500, 64, 4)
        h.route(x, r)
        want.append([t.clone() for t in r])
    static, out = xs[0].clone(), fresh(gm, 500, 64, 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        h.route(static, out)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            h.route(static, out)
    torch.cuda.synchronize()
    for x, w in zip(xs, want):
        static.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, w):
            assert torch.equal(a, b)
    outs = [fresh(gm, 500, 64, 4) for _ in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for x, o, s in zip(xs, outs, streams):
            h.route(x, o, stream=s)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        for a, b in zip(o, w):
            assert torch.equal(a, b)


def test_first_call_may_be_captured(gm):
    x = torch.randn((300, 32), generator=torch.Generator().manual_seed(20)).cuda()
    with gm.Gemm(0) as h:
        out = fresh(gm, 300, 32, 2)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            h.route(x, out)
        graph.replay()
        torch.cuda.synchronize()
        _, e = definition(x, 2)
        assert torch.equal(out.expert.cpu(), e)
        check_sorted(out, 32)


def test_refusals(gm, h):
    x = torch.zeros((4, 8), device="cuda")
    good = gm.routing_empty(4, 8, 2)
    with pytest.raises(gm.GemmError, match="divide"):
        h.route(x, good, groups=3)
    with pytest.raises(ValueError, match="bias"):
        h.route(x, good, bias=torch.zeros(7, device="cuda"))
    with pytest.raises(ValueError, match="out.order"):
        h.route(x, good._replace(order=good.order[:7]))
    with pytest.raises(ValueError, match="out.expert"):
        h.route(x, good._replace(expert=good.expert.int()))
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        h.route(x.half(), good)
    with pytest.raises(ValueError, match="overlap"):
        h.route(x[:1].expand(4, 8), good)
    with pytest.raises(ValueError, match="dlogits"):
        h.route_grad(x, good.expert, good.weights, x.bfloat16())


def test_routed_rows_through_the_grouped_product(gm):
    """The router's order and offsets as grouped_matmul takes them, padding
    included: every choice's row is its token times its expert's matrix."""
    from dense_gemm_sm100_gb300.experts import grouped_matmul, route
    gen = torch.Generator().manual_seed(21)
    T, E, k, K, N = 90, 12, 3, 64, 40
    logits = draw_logits(T, E, torch.float32, 22).cuda().requires_grad_()
    x = torch.randint(-2, 3, (T, K), generator=gen).bfloat16().cuda()
    w = torch.randint(-2, 3, (E, K, N), generator=gen).bfloat16().cuda().requires_grad_()
    r = route(logits, k)
    y = grouped_matmul(x[r.order // k], w, r.offsets, "row", torch.float32)
    flat = r.expert.flatten()[r.order]
    want = torch.einsum("rk,rkn->rn", x[r.order // k].float(), w.detach()[flat.clamp(min=0)].float())
    want[flat < 0] = 0
    assert torch.equal(y, want)
    (y * r.weights.flatten()[r.order, None]).square().sum().backward()
    assert torch.isfinite(logits.grad).all() and (logits.grad[T // 2] == 0).all()
    assert (w.grad != 0).any()
