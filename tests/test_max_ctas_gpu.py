"""GEMM_OPT_MAX_CTAS in the router, the 8-bit products and conversions and the
orthogonalised update: the same bits from few CTAs, and no more of them than
allowed.  A launch confined to one CTA has one of 152 SMs; work that takes all of
them a few microseconds at the memory's rate then takes far more than five times
as long (an SM alone reads at about 1/60 of it)."""
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


@pytest.fixture()
def h(gm):
    with gm.Gemm(0) as handle:
        yield handle


def calls(gm, h, dtype):
    """(name, call) pairs; a call returns what it wrote."""
    gen = torch.Generator().manual_seed(1)
    rand = lambda *s: torch.randn(s, generator=gen).to(dtype).cuda()
    x, w, G = rand(700, 1000), rand(300, 1000), rand(3, 200, 330)
    small, odd = rand(2, 50, 70), rand(1, 130, 65)
    logits, dw = rand(3000, 60), torch.randn((3000, 4), generator=gen).cuda()
    offsets = torch.tensor([0, 250, 250, 700], device="cuda")
    A, B = gm.i8_empty(700, 1000), gm.i8_empty(300, 1000)
    h.i8_quantise(x, A)
    h.i8_quantise(w, B)
    r = gm.routing_empty(3000, 60, 4)
    h.route(logits, r)
    grouped = gm.I8(B.codes, B.scales, 1000)

    def quantised(layout, batch):
        src = x.view(7, 100, 1000) if batch else x
        rows, K = (700, 1000) if layout == "col" else (7000 if batch else 1000, 100 if batch else 700)
        q = gm.i8_empty(rows, K)
        q.codes.fill_(99)
        h.i8_quantise(src, q, layout)
        return q.codes, q.scales

    def wide():
        src = x.view(-1)[:43 * 16000].view(43, 16000)
        q = gm.i8_empty(43, 16000)
        h.i8_quantise(src, q)
        return q.codes, q.scales

    def dequantised():
        out = torch.empty((700, 1000), dtype=dtype, device="cuda")
        return h.i8_dequantise(A, out),

    def product(rows):
        a = gm.I8(A.codes[:rows], A.scales[:rows], 1000)
        return h.run_i8(a, B, torch.empty((rows, 300), dtype=dtype, device="cuda")),

    def grouped_product(rows):
        a = gm.I8(A.codes[:rows], A.scales[:rows], 1000)
        bounds = (offsets * rows) // 700
        return h.run_i8_grouped(a, grouped, bounds, torch.zeros((rows, 100), dtype=dtype, device="cuda")),

    def routed():
        out = gm.routing_empty(3000, 60, 4)
        h.route(logits, out)
        return tuple(out)

    def gradient(renormalise):
        return h.route_grad(logits, r.expert, dw, torch.empty_like(logits), renormalise=renormalise),

    return [("columns", lambda: quantised("col", False)), ("columns of a batch", lambda: quantised("col", True)),
            ("rows", lambda: quantised("row", False)), ("rows of a batch", lambda: quantised("row", True)),
            ("wide rows", wide), ("dequantised", dequantised), ("few rows", lambda: product(4)),
            ("eight rows", lambda: product(8)), ("product", lambda: product(700)),
            ("few rows a group", lambda: grouped_product(6)), ("grouped", lambda: grouped_product(700)),
            ("routed", routed), ("gradient", lambda: gradient(True)), ("gradient of the row", lambda: gradient(False)),
            ("update", lambda: (h.orthogonalise(G, torch.empty_like(G)),)),
            ("turned", lambda: (h.orthogonalise(odd, torch.empty_like(odd)),)),
            ("small updates", lambda: (h.orthogonalise(small, torch.empty_like(small)),))]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_few_ctas_give_the_same_bits(gm, h, dtype):
    todo = calls(gm, h, dtype)
    want = [[t.clone() for t in call()] for _, call in todo]
    # tiles are chosen by the CTAs there are; these products' sums do not depend on them
    for most in (1, 2, 3, 7):
        h.set_option(gm.GEMM_OPT_MAX_CTAS, most)
        for (name, call), w in zip(todo, want):
            if name in ("product", "grouped", "update", "turned", "small updates"):
                continue
            got = call()
            h.sync_status()
            assert all(torch.equal(a, b) for a, b in zip(got, w)), (name, most)
    for tile, names in ((1032, ("product", "grouped")), (1064, ("update", "turned", "small updates"))):
        h.set_option(gm.GEMM_OPT_GROUPED_TILE, 1032)
        h.set_option(gm.GEMM_OPT_ORTHO_TILE, 1064)
        for name, call in todo:
            if name not in names:
                continue
            h.set_option(gm.GEMM_OPT_MAX_CTAS, 0)
            w = [t.clone() for t in call()]
            for most in (1, 2, 7):
                h.set_option(gm.GEMM_OPT_MAX_CTAS, most)
                got = call()
                h.sync_status()
                assert all(torch.equal(a, b) for a, b in zip(got, w)), (name, most)


def test_the_start_of_many_matrices(gm, h):
    """More than 1024 CTAs' worth: the factors by a launch of their own."""
    G = torch.randn((150, 200, 200), generator=torch.Generator().manual_seed(2)).cuda()
    h.set_option(gm.GEMM_OPT_ORTHO_TILE, 1128)
    want = h.orthogonalise(G, torch.empty_like(G), 1)
    for most in (5, 64):
        h.set_option(gm.GEMM_OPT_MAX_CTAS, most)
        got = h.orthogonalise(G, torch.empty_like(G), 1)
        h.sync_status()
        assert torch.equal(got, want)


def median_us(call):
    call()
    torch.cuda.synchronize()
    times = []
    for _ in range(7):
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        call()
        end.record()
        end.synchronize()
        times.append(start.elapsed_time(end) * 1e3)
    return sorted(times)[3]


@pytest.mark.parametrize("what", ["quantise", "quantise rows", "dequantise", "gradient", "few rows"])
def test_one_cta_takes_one_sm(gm, h, what):
    x = torch.randn((8192, 4096), device="cuda").bfloat16()
    q = gm.i8_empty(8192, 4096)
    turned = gm.i8_empty(4096, 8192)
    h.i8_quantise(x, q)
    a, C = gm.I8(q.codes[:4], q.scales[:4], 4096), torch.empty((4, 8192), device="cuda")
    logits = torch.randn((65536, 128), device="cuda")
    expert, dw = torch.zeros((65536, 8), dtype=torch.int64, device="cuda"), torch.ones((65536, 8), device="cuda")
    d = torch.empty_like(logits)
    call = {"quantise": lambda: h.i8_quantise(x, q), "quantise rows": lambda: h.i8_quantise(x, turned, "row"),
            "dequantise": lambda: h.i8_dequantise(q, x), "few rows": lambda: h.run_i8(a, q, C),
            "gradient": lambda: h.route_grad(logits, expert, dw, d)}[what]
    free = median_us(call)
    h.set_option(gm.GEMM_OPT_MAX_CTAS, 1)
    assert median_us(call) > 5 * free
