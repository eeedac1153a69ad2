"""Measured cases of the expert router, the 8-bit integer products and the orthogonalised
update.

Operators, by the ``op`` of a case:

``route``        logits of a router -> every token's k experts and their weights, and the
                 rows (token, choice) sorted by expert with the experts' offsets, as the
                 grouped products take them.
``route_grad``   the same, and the gradient of the logits for a gradient of the weights.
``i8_product``   Y = (Q(X) · Wq^T) with 8-bit integers: activations quantised on the way in
                 with one scale a token, weights held with one scale a channel.
``i8_grouped``   the same with one 8-bit weight matrix per expert and ragged groups.
``ortho``        the orthogonal factor of an update by Newton-Schulz steps: X = G / |G|,
                 then X <- a X + (b A + c A^2) X with A = X X^T, on the smaller side.

``own`` chooses between the plain form (elementary torch operations in 32 bits, 64 where a
choice or a long sum needs them) and the library's calls.  Both take the state that
``prepare`` makes.
"""
import math

import torch

own = False

COEFFICIENTS = (3.4445, -4.7750, 2.0315)
STEPS = 5
EPS = 1e-7
TINY = 1e-20  # added to the sum of sigmoid scores

# --------------------------------------------------------------------- cases


def listed():
    return [
        # one decoding step of a 16-row batch: latency
        _route("route_decode", 16, 64, 8, "softmax", "f32"),
        # a prompt of 16384 tokens over 256 experts in 8 groups, balanced by a bias
        _route("route_prompt", 16384, 256, 8, "sigmoid", "f32", bias=True, groups=8, top_groups=4, scale=2.5),
        # a padded training batch of odd sizes, BF16 logits, weights not renormalised
        _route("route_grad_odd", 1357, 60, 4, "softmax", "bf16", op="route_grad", renormalise=False, padded=0.2),
        # a training step of 32768 tokens
        _route("route_grad_train", 32768, 128, 8, "softmax", "bf16", op="route_grad"),
        # decoding with 8-bit weights: 4 rows, feed-forward shape
        _i8("i8_decode", 4, 4096, 14336, "bf16"),
        # a short prompt, odd sizes, FP32 results
        _i8("i8_odd", 301, 1000, 2047, "f32"),
        # a prompt of 8192 rows, the feed-forward shape
        _i8("i8_ffn", 8192, 4096, 14336, "bf16"),
        # decoding over 128 small experts
        _i8g("i8_grouped_decode", 32, 128, 2048, 2048, "bf16"),
        # a ragged prompt over 32 experts, odd output width
        _i8g("i8_grouped_prompt", 12001, 32, 4096, 2815, "bf16"),
        # the update of one small matrix: latency
        _ortho("ortho_small", 1, 256, 384, "bf16"),
        # the updates of 13 small experts in FP32, odd sizes
        _ortho("ortho_f32_odd", 13, 1020, 520, "f32"),
        # the updates of 16 experts of a training step
        _ortho("ortho_experts", 16, 4096, 2048, "bf16"),
    ]


def _route(name, rows, experts, k, scoring, dtype, op="route", bias=False, groups=1, top_groups=1, renormalise=True,
           scale=1.0, padded=0.0):
    return {"name": name, "op": op, "rows": rows, "experts": experts, "k": k, "scoring": scoring, "dtype": dtype,
            "bias": bias, "groups": groups, "top_groups": top_groups, "renormalise": renormalise, "scale": scale,
            "padded": padded}


def _i8(name, rows, K, N, out):
    return {"name": name, "op": "i8_product", "rows": rows, "K": K, "N": N, "out": out}


def _i8g(name, rows, experts, K, N, out):
    return {"name": name, "op": "i8_grouped", "rows": rows, "experts": experts, "K": K, "N": N, "out": out}


def _ortho(name, batch, rows, cols, dtype):
    return {"name": name, "op": "ortho", "batch": batch, "rows": rows, "cols": cols, "dtype": dtype}


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def width(lo, hi):  # odd sizes, multiples of 8 and round sizes in turn
        v = log_int(lo, hi)
        step = rng.choice([1, 8, 8, 64, 64, 256])
        return max(lo, v // step * step)

    top = max(work(c)["flops"] for c in listed())
    top_bytes = max(work(c)["bytes"] for c in listed())
    while True:
        op = rng.choice(["route", "route_grad", "i8_product", "i8_grouped", "ortho", "ortho"])
        if op in ("route", "route_grad"):
            groups = rng.choice([1, 1, 2, 4, 8])
            experts = groups * log_int(4, 384 // groups)
            top_groups = rng.randint(1, groups)
            k = rng.randint(1, min(8, top_groups * (experts // groups)))
            scoring = rng.choice(["softmax", "sigmoid"])
            c = _route("", log_int(1, 32768), experts, k, scoring, rng.choice(["f32", "bf16"]), op,
                       bias=scoring == "sigmoid" and rng.random() < 0.7, groups=groups, top_groups=top_groups,
                       renormalise=k > 1 and rng.random() < 0.7, scale=rng.choice([1.0, 2.5]),
                       padded=rng.choice([0.0, 0.0, 0.3]))
        elif op == "ortho":
            batch = log_int(1, 16)
            c = _ortho("", batch, width(32, 4096), width(32, 4096), rng.choice(["bf16", "bf16", "f32"]))
        else:
            rows, K, N = log_int(1, 16384), width(256, 8192), width(256, 14336)
            out = rng.choice(["bf16", "f32"])
            c = _i8("", rows, K, N, out) if op == "i8_product" else _i8g("", rows, log_int(1, 128), K, N, out)
        del c["name"]
        w = work(c)
        if w["flops"] <= top and w["bytes"] <= top_bytes:
            return c


# --------------------------------------------------------------------- inputs

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _sizes(case, seed):
    """Rows of each group: multinomial draws from a router's skewed preferences."""
    gen = torch.Generator().manual_seed(seed * 1000003 + case["rows"])
    pref = torch.exp(0.7 * torch.randn(case["experts"], generator=gen))
    picks = torch.multinomial(pref, case["rows"], replacement=True, generator=gen)
    return torch.bincount(picks, minlength=case["experts"]).tolist()


def _bounds(sizes):
    b = [0]
    for s in sizes:
        b.append(b[-1] + s)
    return b


def _activations(gen, rows, K):
    """Normalised activations: unit variance, with the few large channels that hidden
    states have."""
    channel = torch.exp(0.3 * torch.randn(K, generator=gen, device="cuda"))
    channel = torch.where(torch.rand(K, generator=gen, device="cuda") < 0.01, channel * 8, channel)
    return (torch.randn((rows, K), generator=gen, device="cuda") * channel).bfloat16()


def _weights_i8(gen, rows, K):
    """A weight matrix (rows x K) as 8-bit codes at a pitch of whole 16 bytes, and its
    channels' scales, made slab by slab."""
    codes = torch.zeros((rows, (K + 15) // 16 * 16), dtype=torch.int8, device="cuda")
    scales = torch.empty(rows, dtype=torch.float32, device="cuda")
    for r in range(0, rows, 16384):
        w = torch.randn((min(16384, rows - r), K), generator=gen, device="cuda") * 0.02
        q, s = _quantise(w)
        codes[r:r + 16384, :K] = q.to(torch.int8)
        scales[r:r + 16384] = s[:, 0]
    return codes, scales


def _updates(gen, batch, rows, cols, dtype):
    """Momentum of gradients: a few directions that carry most of the norm, and noise."""
    rank = max(2, min(rows, cols) // 8)
    decay = torch.logspace(0, -2, rank, device="cuda")
    left = torch.randn((batch, rows, rank), generator=gen, device="cuda") * decay
    right = torch.randn((batch, rank, cols), generator=gen, device="cuda")
    noise = torch.randn((batch, rows, cols), generator=gen, device="cuda")
    return ((left @ right / rank ** 0.5 + 0.03 * noise) * 1e-3).to(dtype)


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, st = case["op"], {"case": case}
    if op in ("route", "route_grad"):
        T, E = case["rows"], case["experts"]
        prefer = 0.5 * torch.randn(E, generator=gen, device="cuda")
        logits = torch.randn((T, E), generator=gen, device="cuda") + prefer
        if case["padded"]:  # tokens of padding may go nowhere
            logits[torch.rand(T, generator=gen, device="cuda") < case["padded"]] = -math.inf
        st["logits"] = logits.to(_TYPES[case["dtype"]])
        st["bias"] = 0.05 * torch.randn(E, generator=gen, device="cuda") if case["bias"] else None
        if op == "route_grad":
            st["dweights"] = torch.randn((T, case["k"]), generator=gen, device="cuda")
    elif op == "ortho":
        st["X"] = _updates(gen, case["batch"], case["rows"], case["cols"], _TYPES[case["dtype"]])
    else:
        st["X"] = _activations(gen, case["rows"], case["K"])
        if op == "i8_grouped":
            st["bounds"] = _bounds(_sizes(case, seed))
            st["offsets"] = torch.tensor(st["bounds"], dtype=torch.int64, device="cuda")
        st["codes"], st["scales"] = _weights_i8(gen, case.get("experts", 1) * case["N"], case["K"])
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    if own:
        from dense_gemm_sm100_gb300 import gemm
        op = case["op"]
        st["handle"] = gemm.Gemm(torch.cuda.current_device())
        if op in ("route", "route_grad"):
            T, E, k = case["rows"], case["experts"], case["k"]
            st["out"] = gemm.routing_empty(T, E, k)
            if op == "route_grad":
                st["dlogits"] = torch.empty_like(st["logits"])
        elif op == "ortho":
            st["O"] = torch.empty_like(st["X"])
        else:
            st["Xq"] = gemm.i8_empty(case["rows"], case["K"])
            st["Wq"] = gemm.I8(st["codes"], st["scales"], case["K"])
            st["Y"] = torch.empty((case["rows"], case["N"]), dtype=_TYPES[case["out"]], device="cuda")
    return st


# ----------------------------------------------------------------------- run


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(st):
    case, h = st["case"], st["handle"]
    op = case["op"]
    if op in ("route", "route_grad"):
        r = h.route(st["logits"], st["out"], case["scoring"], st["bias"], case["groups"], case["top_groups"],
                    case["renormalise"], case["scale"])
        if op == "route":
            return r.weights, r.expert, r.order, r.offsets
        h.route_grad(st["logits"], r.expert, st["dweights"], st["dlogits"], case["scoring"], case["renormalise"],
                     case["scale"])
        return r.weights, r.expert, r.order, r.offsets, st["dlogits"]
    if op == "ortho":
        return h.orthogonalise(st["X"], st["O"], STEPS, COEFFICIENTS, EPS)
    h.i8_quantise(st["X"], st["Xq"])
    if op == "i8_product":
        return h.run_i8(st["Xq"], st["Wq"], st["Y"])
    return h.run_i8_grouped(st["Xq"], st["Wq"], st["offsets"], st["Y"])


def _run_plain(st):
    case = st["case"]
    op = case["op"]
    if op in ("route", "route_grad"):
        return _route_plain(st)
    if op == "ortho":
        return _ortho_plain(st["X"])
    K, N, out = case["K"], case["N"], _TYPES[case["out"]]
    q, s = _quantise(st["X"])
    if op == "i8_product":
        return ((q @ st["codes"][:, :K].float().t()) * s * st["scales"]).to(out)
    b = st["bounds"]
    y = [q[b[g]:b[g + 1]] @ st["codes"][g * N:(g + 1) * N, :K].float().t() * st["scales"][g * N:(g + 1) * N]
         for g in range(case["experts"]) if b[g + 1] > b[g]]
    return (torch.cat(y) * s).to(out)


def _quantise(x):
    """Whole numbers in -127..127 (in 32-bit floating point) and one scale a row: the scale is
    max|x| / 127 in FP32, the numbers x / scale rounded to nearest, ties to even.  The quotient
    is taken in 64 bits, where none that is not a tie rounds to one."""
    s = (x.float().abs().amax(-1, keepdim=True).double() / 127).float()
    q = torch.round(x.double() / s.double()).clamp(-127, 127)
    return torch.where(s > 0, q, torch.zeros_like(q)).float(), s


def _route_plain(st):
    """The ranking is by logits; where a bias or groups come in, by scores in 64 bits, so that
    no rounding decides.  Logits of minus infinity are no choice (expert -1, weight 0)."""
    case = st["case"]
    logits, bias, k, groups = st["logits"].float(), st["bias"], case["k"], case["groups"]
    T, E = logits.shape
    soft, open_ = case["scoring"] == "softmax", logits > -math.inf
    rank = logits.double()
    if bias is not None or groups > 1:
        if soft:
            rank = torch.exp(rank - rank.amax(-1, keepdim=True).clamp(min=-3e38))
            rank = rank / rank.sum(-1, keepdim=True)
        else:
            rank = 1 / (1 + torch.exp(-rank))
        if bias is not None:
            rank = rank + bias.double()
        rank = torch.where(open_, rank, -math.inf)
    if groups > 1:
        best = torch.sort(rank.view(T, groups, -1), -1, descending=True)[0][..., :2]
        second = best[..., 1:].sum(-1)
        score = best[..., 0] + torch.where(second > -math.inf, second, torch.zeros_like(second))
        at = torch.sort(score, dim=-1, descending=True, stable=True)[1][:, :case["top_groups"]]
        kept = torch.zeros((T, groups), dtype=torch.bool, device=logits.device).scatter_(1, at, True)
        rank = torch.where(kept.repeat_interleave(E // groups, 1), rank, -math.inf)
    value, expert = torch.sort(rank, dim=-1, descending=True, stable=True)
    chosen = value[:, :k] > -math.inf
    index = expert[:, :k]
    expert = torch.where(chosen, index, -1)
    picked = torch.gather(logits, 1, index)
    zero = torch.zeros_like(picked)
    if soft:
        top = logits.amax(-1, keepdim=True).clamp(min=-3e38)
        e = torch.exp(logits - top)
        score = e / e.sum(-1, keepdim=True).clamp(min=1e-30)
        top = torch.where(chosen, picked, -math.inf).amax(-1, keepdim=True).clamp(min=-3e38)
        share = torch.where(chosen, torch.exp(picked - top), zero)
    else:
        score = 1 / (1 + torch.exp(-logits))
        share = torch.where(chosen, torch.gather(score, 1, index), zero)
    own_score = torch.where(chosen, torch.gather(score, 1, index), zero)
    total = share.sum(-1, keepdim=True)
    total = total + TINY if not soft else total.clamp(min=1e-30)
    weights = case["scale"] * (share / total if case["renormalise"] else own_score)
    flat = expert.flatten()
    by_expert, order = torch.sort(flat, stable=True)
    offsets = torch.searchsorted(by_expert, torch.arange(E + 1, device=flat.device))
    if case["op"] == "route":
        return weights, expert, order, offsets
    g = torch.where(chosen, st["dweights"] * case["scale"], zero)
    dlogits = torch.zeros_like(logits)
    if soft and case["renormalise"]:
        w = share / total
        dlogits.scatter_add_(1, index, w * (g - (w * g).sum(-1, keepdim=True)))
    elif soft:
        dlogits.scatter_add_(1, index, own_score * g)
        dlogits -= score * (own_score * g).sum(-1, keepdim=True)
    else:
        if case["renormalise"]:
            g = (g - (share / total * g).sum(-1, keepdim=True)) / total
        # 1 - sigmoid(x) = sigmoid(-x), without the cancellation
        dlogits.scatter_add_(1, index, torch.where(chosen, g * own_score / (1 + torch.exp(picked)), zero))
    return weights, expert, order, offsets, dlogits.to(st["logits"].dtype)


def _ortho_plain(G):
    a, b, c = COEFFICIENTS
    tall = G.shape[1] > G.shape[2]
    X = G.float().transpose(1, 2) if tall else G.float()
    norm = G.double().square().sum((1, 2), keepdim=True).sqrt()  # a long sum
    X = X / (norm + EPS).float()
    for _ in range(STEPS):
        A = X @ X.transpose(1, 2)
        X = a * X + (b * A + c * (A @ A)) @ X
    return (X.transpose(1, 2) if tall else X).to(G.dtype).contiguous()


# ---------------------------------------------------------------------- work


def work(case):
    """Bytes and operations of one pass: every input read once (the weights of experts that
    have rows), every output written once; symmetric products count half."""
    op = case["op"]
    if op in ("route", "route_grad"):
        T, E, k = case["rows"], case["experts"], case["k"]
        es = 2 if case["dtype"] == "bf16" else 4
        there = T * E * es + T * k * (4 + 8 + 8) + (E + 1) * 8 + (4 * E if case["bias"] else 0)
        back = T * E * es + T * k * 4 if op == "route_grad" else 0
        return {"bytes": there + back, "flops": T * E * (4 if op == "route" else 8)}
    if op == "ortho":
        m, n = sorted((case["rows"], case["cols"]))
        es = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2 * case["batch"] * m * n * es, "flops": case["batch"] * STEPS * (3 * m * m * n + m ** 3)}
    rows, K, N = case["rows"], case["K"], case["N"]
    busy = sum(1 for s in _sizes(case, 0) if s) if op == "i8_grouped" else 1
    eo = 2 if case["out"] == "bf16" else 4
    return {"bytes": rows * K * 2 + busy * N * (K + 4) + rows * N * eo, "flops": 2 * rows * K * N}


# --------------------------------------------------------------------- exact


def _exact_codes(x):
    """Codes and scales in 64 bits: the integer next to x / scale, found from below."""
    x = x.double()
    scale = torch.div(x.abs().max(dim=1).values, 127).float().double()[:, None]
    size = x.abs() / torch.where(scale == 0, 1.0, scale)
    low = torch.floor(size)
    part = size - low
    up = (part > 0.5) | ((part == 0.5) & (low % 2 == 1))
    return torch.sign(x) * (low + up).clamp(max=127) * (scale > 0), scale


def _exact_route(st):
    case = st["case"]
    out = []
    top, k, G = case["scale"], case["k"], case["groups"]
    bias = st["bias"].double() if st["bias"] is not None else 0.0
    for n, x in enumerate(st["logits"].double().split(1024)):
        T, E = x.shape
        live = torch.isfinite(x)
        if case["scoring"] == "softmax":
            p = torch.where(live, torch.softmax(torch.where(live, x, -1e4), 1), 0.0)
        else:
            p = torch.where(live, torch.sigmoid(x), 0.0)
        c = p + bias if (st["bias"] is not None or G > 1) else x

        def places(v, ok):  # how many come before each
            before = (v[:, None, :] > v[:, :, None]) & ok[:, None, :]
            same = (v[:, None, :] == v[:, :, None]) & ok[:, None, :]
            idx = torch.arange(v.shape[1], device=v.device)
            return (before | (same & (idx[None, :] < idx[:, None]))).sum(2)

        ok = live
        if G > 1:
            each = E // G
            inside = places(c.reshape(T * G, each), live.reshape(T * G, each))
            two = (inside < 2) & live.reshape(T * G, each)
            total = (c.reshape(T * G, each) * two).sum(1).view(T, G)
            some = live.view(T, G, each).any(2)
            keep = (places(total, some) < case["top_groups"]) & some
            ok = live & keep[:, :, None].expand(T, G, each).reshape(T, E)
        place = places(c, ok)
        sel = ok & (place < k)
        if case["renormalise"]:
            total = (p * sel).sum(1, keepdim=True)
            w = p / (total + (TINY if case["scoring"] == "sigmoid" else 0.0)).clamp(min=1e-300)
        else:
            w = p
        slot = torch.where(sel, place, k)
        weights = torch.zeros((T, k + 1), dtype=torch.float64, device=x.device)
        weights.scatter_(1, slot, torch.where(sel, top * w, 0.0))
        if case["op"] == "route":
            out.append((weights[:, :k],))
            continue
        dw = torch.zeros((T, k + 1), dtype=torch.float64, device=x.device)
        dw[:, :k] = st["dweights"][n * 1024:n * 1024 + 1024].double()
        g = torch.where(sel, top * torch.gather(dw, 1, slot), 0.0)  # by expert
        if case["renormalise"]:
            total = (p * sel).sum(1, keepdim=True) + (TINY if case["scoring"] == "sigmoid" else 0.0)
            dp = torch.where(sel, (g - (g * p).sum(1, keepdim=True) / total.clamp(min=1e-300)) / total.clamp(min=1e-300), 0.0)
        else:
            dp = g
        if case["scoring"] == "softmax":
            dx = p * (dp - (p * dp).sum(1, keepdim=True))
        else:
            dx = dp * p * torch.sigmoid(-x)
        out.append((weights[:, :k], torch.where(live, dx, 0.0)))
    weights = torch.cat([o[0] for o in out])
    return (weights, None, None, None) + ((torch.cat([o[1] for o in out]),) if case["op"] == "route_grad" else ())


def _exact_ortho(G):
    a, b, c = COEFFICIENTS
    out = []
    for M in G.double():
        M = M / (torch.linalg.vector_norm(M) + EPS)
        wide = M.shape[0] <= M.shape[1]
        for _ in range(STEPS):
            S = torch.mm(M, M.T) if wide else torch.mm(M.T, M)
            P = torch.addmm(S, S, S, beta=b, alpha=c)
            P.diagonal().add_(a)
            M = torch.mm(P, M) if wide else torch.mm(M, P)
        out.append(M)
    return torch.stack(out)


def exact(case, seed):
    st = _inputs(case, seed)
    op = case["op"]
    if op in ("route", "route_grad"):
        return _exact_route(st)
    if op == "ortho":
        return _exact_ortho(st["X"])
    K, N = case["K"], case["N"]
    codes, scale = _exact_codes(st["X"])
    if op == "i8_product":
        return torch.einsum("rk,nk->rn", codes * scale, st["codes"][:, :K].double() * st["scales"].double()[:, None])
    parts, ends = [], st["bounds"]
    for g, (lo, hi) in enumerate(zip(ends[:-1], ends[1:])):
        if hi > lo:
            w = st["codes"][g * N:g * N + N, :K].double() * st["scales"][g * N:g * N + N].double()[:, None]
            parts.append(torch.einsum("rk,nk->rn", codes[lo:hi] * scale[lo:hi], w))
    return torch.cat(parts)
