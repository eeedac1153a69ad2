"""Measured cases of the expert products and of the microscaled 4-bit operators.

Operators, by the ``op`` of a case:

``grouped``      Y[r] = X[r] · W[e(r)]: rows sorted by expert, ragged groups given by
                 offsets on the device (the forward pass of an expert layer).
``grouped_grad`` its two gradients: dX[r] = dY[r] · W[e(r)]^T and dW[e] = X_e^T · dY_e
                 (a group without rows has dW[e] = 0).
``mx4_round``    x -> microscaled 4-bit floating point (E2M1 elements, one E8M0 scale per
                 32 along the row) and back to the values the codes stand for.
``mx4_product``  Y = Q(X) · Wq^T: activations quantised on the way in, weights held in 4 bits.
``mx4_grouped``  the same with one 4-bit weight matrix per expert and ragged groups.

``own`` chooses between the plain form (elementary torch operations in 32 bits) and the
library's calls.  Both take the state that ``prepare`` makes.
"""
import math

import torch

own = False

BLOCK = 32  # elements that share a scale

# --------------------------------------------------------------------- cases


def listed():
    return [
        # one decoding step of a 16-row batch over many small experts: latency
        _grouped("grouped_decode", 16, 64, 2048, 1024, "col", "bf16", "bf16"),
        # a short prompt with odd sizes, few rows an expert, FP32 results
        _grouped("grouped_odd", 1357, 24, 1416, 2047, "col", "bf16", "f32"),
        # a prompt of 8192 rows over 32 experts
        _grouped("grouped_prompt", 8192, 32, 4096, 2048, "row", "bf16", "bf16"),
        # a long batch over 8 experts of the feed-forward shape 4096 x 14336
        _grouped("grouped_large", 16384, 8, 4096, 14336, "row", "bf16", "bf16"),
        # both gradients of a small layer in TF32, odd sizes
        _grad("grad_tf32_odd", 2011, 13, 520, 1020, "col", "tf32"),
        # both gradients of a training step in BF16 (dW kept in FP32)
        _grad("grad_train", 8192, 16, 4096, 2048, "row", "bf16"),
        # a few activations rounded to 4 bits, a row that ends inside a block
        _round("mx4_round_small", 33, 1000, "bf16"),
        # a weight or activation matrix of a large layer rounded to 4 bits
        _round("mx4_round_large", 16384, 8192, "bf16"),
        # decoding with 4-bit weights: 4 rows, feed-forward shape
        _mx4("mx4_decode", 4, 4096, 14336, "bf16"),
        # a prompt of 8192 rows, the feed-forward shape
        _mx4("mx4_ffn", 8192, 4096, 14336, "bf16"),
        # decoding over 128 small experts with 4-bit weights
        _mx4g("mx4_grouped_decode", 32, 128, 2048, 2048, "bf16"),
        # a ragged prompt over 32 experts with 4-bit weights, odd output width
        _mx4g("mx4_grouped_prompt", 12001, 32, 4096, 2815, "bf16"),
    ]


def _grouped(name, rows, groups, K, N, layout, dtype, out):
    return {"name": name, "op": "grouped", "rows": rows, "groups": groups, "K": K, "N": N,
            "layout": layout, "dtype": dtype, "out": out}


def _grad(name, rows, groups, K, N, layout, dtype):
    return {"name": name, "op": "grouped_grad", "rows": rows, "groups": groups, "K": K, "N": N,
            "layout": layout, "dtype": dtype}


def _round(name, rows, K, dtype):
    return {"name": name, "op": "mx4_round", "rows": rows, "K": K, "dtype": dtype}


def _mx4(name, rows, K, N, out):
    return {"name": name, "op": "mx4_product", "rows": rows, "K": K, "N": N, "out": out}


def _mx4g(name, rows, groups, K, N, out):
    return {"name": name, "op": "mx4_grouped", "rows": rows, "groups": groups, "K": K, "N": N, "out": out}


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
        op = rng.choice(["grouped", "grouped", "grouped_grad", "grouped_grad", "mx4_round", "mx4_product",
                         "mx4_grouped"])
        rows, groups = log_int(1, 16384), log_int(1, 128)
        K, N = width(256, 8192), width(256, 14336)
        if op == "grouped":
            dtype = rng.choice(["bf16", "bf16", "tf32"])
            out = "f32" if dtype == "tf32" else rng.choice(["bf16", "f32"])
            c = _grouped("", rows, groups, K, N, rng.choice(["row", "col"]), dtype, out)
        elif op == "grouped_grad":
            c = _grad("", max(rows, 64), min(groups, 32), K, N, rng.choice(["row", "col"]),
                      rng.choice(["bf16", "bf16", "tf32"]))
        elif op == "mx4_round":
            c = _round("", rows, K, rng.choice(["bf16", "f32"]))
        elif op == "mx4_product":
            c = _mx4("", rows, K, N, rng.choice(["bf16", "f32"]))
        else:
            c = _mx4g("", rows, groups, K, N, rng.choice(["bf16", "f32"]))
        del c["name"]
        w = work(c)
        if 3072 not in (K, N, rows) and w["flops"] <= top and w["bytes"] <= top_bytes:
            return c


# --------------------------------------------------------------------- inputs

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "tf32": torch.float32}


def _sizes(case, seed):
    """Rows of each group: multinomial draws from a router's skewed preferences."""
    gen = torch.Generator().manual_seed(seed * 1000003 + case["rows"])
    pref = torch.exp(0.7 * torch.randn(case["groups"], generator=gen))
    picks = torch.multinomial(pref, case["rows"], replacement=True, generator=gen)
    return torch.bincount(picks, minlength=case["groups"]).tolist()


def _bounds(sizes):
    b = [0]
    for s in sizes:
        b.append(b[-1] + s)
    return b


def _normal(gen, shape, sigma, dtype):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * sigma).to(dtype)


def _activations(gen, rows, K, dtype):
    """Normalised activations: unit variance, with the few large channels that hidden
    states have."""
    channel = torch.exp(0.3 * torch.randn(K, generator=gen, device="cuda"))
    channel = torch.where(torch.rand(K, generator=gen, device="cuda") < 0.01, channel * 8, channel)
    return (torch.randn((rows, K), generator=gen, device="cuda") * channel).to(dtype)


def _ceil_to(x, m):
    return (x + m - 1) // m * m


def _pack(values, exps, K):
    """Codes two to a byte (even element in the low half) and scale bytes, rows padded to
    whole blocks and pitches to 16 bytes."""
    rows, Kp = values.shape[0], _ceil_to(K, BLOCK)
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=values.device)
    code = torch.searchsorted(grid, values.abs()) + 8 * torch.signbit(values)
    code = code.to(torch.uint8)
    codes = torch.zeros((rows, _ceil_to(Kp // 2, 16)), dtype=torch.uint8, device=values.device)
    codes[:, :Kp // 2] = code[:, 0::2] | (code[:, 1::2] << 4)
    scales = torch.zeros((rows, _ceil_to(Kp // BLOCK, 16)), dtype=torch.uint8, device=values.device)
    scales[:, :Kp // BLOCK] = (exps + 127).to(torch.uint8)
    return codes, scales


def _weights_mx4(gen, rows, K):
    """A weight matrix (rows x K) as codes and scales, made slab by slab."""
    parts = []
    for r in range(0, rows, 32768):
        w = torch.randn((min(32768, rows - r), K), generator=gen, device="cuda") * 0.02
        parts.append(_pack(*_quantise(w), K))
    return torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, rows, K = case["op"], case["rows"], case["K"]
    st = {"case": case}
    if "groups" in case:
        sizes = _sizes(case, seed)
        st["bounds"] = _bounds(sizes)
        st["offsets"] = torch.tensor(st["bounds"], dtype=torch.int64, device="cuda")
    if op in ("grouped", "grouped_grad"):
        dt, N = _TYPES[case["dtype"]], case["N"]
        st["X"] = _activations(gen, rows, K, dt)
        shape = (K, N) if case["layout"] == "row" else (N, K)
        st["W"] = torch.stack([_normal(gen, shape, 0.02, dt) for _ in range(case["groups"])])
        if op == "grouped_grad":
            st["dY"] = _normal(gen, (rows, N), 0.01, dt)
    elif op == "mx4_round":
        st["X"] = _activations(gen, rows, K, _TYPES[case["dtype"]])
    else:
        st["X"] = _activations(gen, rows, K, torch.bfloat16)
        st["codes"], st["scales"] = _weights_mx4(gen, case.get("groups", 1) * case["N"], K)
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    if own:
        from dense_gemm_sm100_gb300 import gemm
        op, rows, K = case["op"], case["rows"], case["K"]
        st["handle"] = gemm.Gemm(torch.cuda.current_device())
        if op == "grouped":
            st["Y"] = torch.empty((rows, case["N"]), dtype=_TYPES[case["out"]], device="cuda")
        elif op == "grouped_grad":
            st["dX"] = torch.empty_like(st["X"])
            st["dW"] = torch.empty(st["W"].shape, dtype=torch.float32, device="cuda")
        else:
            st["Xq"] = gemm.mx4_empty(rows, K)
            if op == "mx4_round":
                st["Y"] = torch.empty_like(st["X"])
            else:
                st["Wq"] = gemm.Mx4(st["codes"], st["scales"], K)
                st["Y"] = torch.empty((rows, case["N"]), dtype=_TYPES[case["out"]], device="cuda")
    return st


# ----------------------------------------------------------------------- run


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(st):
    case, h = st["case"], st["handle"]
    op = case["op"]
    if op == "grouped":
        return h.run_grouped(st["X"], st["W"], st["offsets"], st["Y"], case["layout"], case["dtype"])
    if op == "grouped_grad":
        flip = "col" if case["layout"] == "row" else "row"
        h.run_grouped(st["dY"], st["W"], st["offsets"], st["dX"], flip, case["dtype"])
        left, right = (st["X"], st["dY"]) if case["layout"] == "row" else (st["dY"], st["X"])
        h.run_grouped_wgrad(left, right, st["offsets"], st["dW"], case["dtype"])
        return st["dX"], st["dW"]
    if op == "mx4_round":
        h.mx4_quantise(st["X"], st["Xq"])
        return h.mx4_dequantise(st["Xq"], st["Y"])
    h.mx4_quantise(st["X"], st["Xq"])
    if op == "mx4_product":
        return h.run_mx4(st["Xq"], st["Wq"], st["Y"])
    return h.run_mx4_grouped(st["Xq"], st["Wq"], st["offsets"], st["Y"])


def _operand(t, dtype):
    """The operand as it enters the multiplier, in 32 bits: TF32 keeps the upper 10 of
    FP32's 23 mantissa bits."""
    if dtype == "tf32":
        return (t.view(torch.int32) & -8192).view(torch.float32)
    return t.float()


def _quantise(x):
    """E2M1 values and block exponents of x (rows x K), K padded with zeros to whole blocks.

    The exponent of a block is floor(log2(max|x|)) - 2 (so that the largest element falls in
    [4, 8)); elements are x / 2^exponent rounded to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6,
    ties to the even code, values past 6 to 6."""
    rows, K = x.shape
    pad = _ceil_to(K, BLOCK) - K
    x = torch.nn.functional.pad(x.float(), (0, pad)).view(rows, -1, BLOCK)
    big = x.abs().amax(-1, keepdim=True)
    exps = torch.where(big > 0, torch.frexp(big)[1] - 3, torch.full_like(big, -127, dtype=torch.int32)).clamp(min=-127)
    v = x * _power(-exps)
    a = v.abs()
    q = 0.5 * ((a > 0.25).float() + (a >= 0.75) + (a > 1.25) + (a >= 1.75)) + (a > 2.5) + (a >= 3.5) + 2.0 * (a > 5.0)
    return torch.copysign(q, v).view(rows, -1), exps.view(rows, -1)


def _power(e):
    """2^e as FP32, exactly, for -127 <= e <= 127 (the lowest one is subnormal)."""
    return torch.where(e > -127, (e + 127) << 23, torch.full_like(e, 1 << 22)).view(torch.float32)


def _dequantise(values, exps, K):
    rows = values.shape[0]
    return (values.view(rows, -1, BLOCK) * _power(exps)[..., None]).view(rows, -1)[:, :K]


def _unpack(codes, scales, K):
    Kp = _ceil_to(K, BLOCK)
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    c = codes[:, :Kp // 2]
    values = torch.stack((table[(c & 15).long()], table[(c >> 4).long()]), -1).view(codes.shape[0], Kp)
    return _dequantise(values, scales[:, :Kp // BLOCK].int() - 127, K)


def _run_plain(st):
    case = st["case"]
    op, K = case["op"], case["K"]
    if op == "mx4_round":
        return _dequantise(*_quantise(st["X"]), K).to(st["X"].dtype)
    if op == "mx4_product":
        x = _dequantise(*_quantise(st["X"]), K)
        return (x @ _unpack(st["codes"], st["scales"], K).t()).to(_TYPES[case["out"]])
    b, N = st["bounds"], case["N"]
    spans = [(g, b[g], b[g + 1]) for g in range(case["groups"]) if b[g + 1] > b[g]]
    if op == "mx4_grouped":
        x = _dequantise(*_quantise(st["X"]), K)
        y = torch.empty((case["rows"], N), dtype=torch.float32, device=x.device)
        for g, lo, hi in spans:
            w = _unpack(st["codes"][g * N:(g + 1) * N], st["scales"][g * N:(g + 1) * N], K)
            y[lo:hi] = x[lo:hi] @ w.t()
        return y.to(_TYPES[case["out"]])
    row, dtype = case["layout"] == "row", case["dtype"]
    X = _operand(st["X"], dtype)
    if op == "grouped":
        y = torch.empty((case["rows"], N), dtype=torch.float32, device=X.device)
        for g, lo, hi in spans:
            w = _operand(st["W"][g], dtype)
            y[lo:hi] = X[lo:hi] @ (w if row else w.t())
        return y.to(_TYPES[case["out"]])
    dY = _operand(st["dY"], dtype)
    dX = torch.empty((case["rows"], K), dtype=torch.float32, device=X.device)
    dW = torch.zeros(st["W"].shape, dtype=torch.float32, device=X.device)
    for g, lo, hi in spans:
        w = _operand(st["W"][g], dtype)
        dX[lo:hi] = dY[lo:hi] @ (w.t() if row else w)
        dW[g] = X[lo:hi].t() @ dY[lo:hi] if row else dY[lo:hi].t() @ X[lo:hi]
    return dX.to(st["X"].dtype), dW


# ---------------------------------------------------------------------- work


def work(case):
    """Bytes and operations of one pass: every input read once (the weights of experts that
    have rows), every output written once."""
    op, rows, K = case["op"], case["rows"], case["K"]
    if op == "mx4_round":
        es = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2 * rows * K * es, "flops": 2 * rows * K}
    N = case["N"]
    busy = sum(1 for s in _sizes(case, 0) if s) if "groups" in case else 1
    if op == "grouped":
        es, eo = (2 if case["dtype"] == "bf16" else 4), (2 if case["out"] == "bf16" else 4)
        return {"bytes": rows * K * es + busy * K * N * es + rows * N * eo, "flops": 2 * rows * K * N}
    if op == "grouped_grad":
        es = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": (2 * rows * K + rows * N + busy * K * N) * es + case["groups"] * K * N * 4,
                "flops": 4 * rows * K * N}
    eo = 2 if case["out"] == "bf16" else 4
    Kp = _ceil_to(K, BLOCK)
    return {"bytes": rows * K * 2 + busy * N * (Kp // 2 + Kp // BLOCK) + rows * N * eo, "flops": 2 * rows * K * N}


# --------------------------------------------------------------------- exact


def _exact_power(p):
    return ((p.long() + 1023) << 52).view(torch.float64)


def _exact_round(x):
    """The 4-bit rounding in 64 bits: the step of |v| in [2^p, 2^(p+1)) is 2^(max(p, 0) - 1)."""
    out = []
    for rows in x.double().split(4096):
        K = rows.shape[1]
        blocks = torch.cat([rows, rows.new_zeros(rows.shape[0], -K % BLOCK)], 1).unflatten(1, (-1, BLOCK))
        top = blocks.abs().max(dim=2, keepdim=True).values
        scale = _exact_power(torch.frexp(top.clamp(min=2.0 ** -125))[1] - 3)
        v = blocks / scale
        step = _exact_power(torch.frexp(v.abs().clamp(min=1.0))[1] - 2)
        q = (torch.round(v / step) * step).clamp(-6, 6)
        out.append((q * scale).flatten(1)[:, :K])
    return torch.cat(out)


def _exact_weights(codes, scales, K):
    half = torch.stack([codes % 16, codes // 16], dim=2).flatten(1)[:, :K].double()
    sign = 1 - 2 * (half >= 8).double()
    low = half % 8
    power = torch.div(low, 2, rounding_mode="floor")
    frac = low % 2
    mag = torch.where(power == 0, frac / 2, (1 + frac / 2) * _exact_power(power - 1))
    scale = _exact_power(scales.double() - 127).repeat_interleave(BLOCK, dim=1)[:, :K]
    return sign * mag * scale


def exact(case, seed):
    st = _inputs(case, seed)
    op, K = case["op"], case["K"]
    if op == "mx4_round":
        return _exact_round(st["X"])
    if op == "mx4_product":
        return _exact_round(st["X"]) @ _exact_weights(st["codes"], st["scales"], K).T
    N, ends = case["N"], st["bounds"]
    starts = list(zip(range(case["groups"]), ends[:-1], ends[1:]))
    if op == "mx4_grouped":
        x = _exact_round(st["X"])
        return torch.cat([x[a:b] @ _exact_weights(st["codes"][g * N:g * N + N], st["scales"][g * N:g * N + N], K).T
                          for g, a, b in starts if b > a])

    def wide(t):
        t = t.double()
        if case["dtype"] != "tf32":
            return t
        m, e = torch.frexp(t)  # 11 significant bits, the rest dropped
        return torch.trunc(m * 2048) / 2048 * _exact_power(e)

    X = wide(st["X"])
    spec = "rk,kn->rn" if case["layout"] == "row" else "rk,nk->rn"
    if op == "grouped":
        return torch.cat([torch.einsum(spec, X[a:b], wide(st["W"][g])) for g, a, b in starts if b > a])
    dY = wide(st["dY"])
    back = "rn,kn->rk" if case["layout"] == "row" else "rn,nk->rk"
    outer = "rk,rn->kn" if case["layout"] == "row" else "rk,rn->nk"
    dX = torch.cat([torch.einsum(back, dY[a:b], wide(st["W"][g])) for g, a, b in starts if b > a])
    dW = torch.stack([torch.einsum(outer, X[a:b], dY[a:b]) for g, a, b in starts])
    return dX, dW
