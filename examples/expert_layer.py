"""A mixture-of-experts feed-forward layer on the grouped products: a few
training steps in BF16, then serving with the experts' weights in microscaled
4-bit floating point.

    python examples/expert_layer.py [--tokens 4096] [--steps 5]

Every token goes to its router's top-k experts; an expert is
down(silu(gate(x)) * up(x)), gate and up held as one column-major matrix.
"""
import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from dense_gemm_sm100_gb300 import gemm  # noqa: E402
from dense_gemm_sm100_gb300.experts import group_rows, grouped_matmul  # noqa: E402


class ExpertLayer(torch.nn.Module):
    def __init__(self, hidden, inner, experts, top_k, device="cuda"):
        super().__init__()
        self.experts, self.top_k = experts, top_k
        def weight(*shape):
            return torch.nn.Parameter((torch.randn(shape, device=device) * shape[-1] ** -0.5).bfloat16())
        self.router = weight(experts, hidden)
        self.gate_up = weight(experts, 2 * inner, hidden)
        self.down = weight(experts, hidden, inner)

    def route(self, x):
        """Chosen experts' weights (tokens, k), the sorted order of the
        (token, choice) rows, and the experts' offsets in it."""
        prob, expert = torch.topk(torch.softmax(x.float() @ self.router.float().t(), -1), self.top_k)
        order, offsets = group_rows(expert.flatten(), self.experts)
        return prob / prob.sum(-1, keepdim=True), order, offsets

    def _combine(self, x, prob, order, y):
        y = y.float() * prob.flatten()[order, None]
        return torch.zeros_like(x, dtype=torch.float32).index_add(0, order // self.top_k, y).to(x.dtype)

    def forward(self, x):
        prob, order, offsets = self.route(x)
        rows = x[order // self.top_k]
        gate, up = grouped_matmul(rows, self.gate_up, offsets, "col").chunk(2, -1)
        y = grouped_matmul(F.silu(gate) * up, self.down, offsets, "col")
        return self._combine(x, prob, order, y)


class ServedExpertLayer:
    """The layer with 4-bit experts: activations are quantised on the way into
    each product."""

    def __init__(self, layer: ExpertLayer, handle: gemm.Gemm):
        self.layer, self.handle = layer, handle
        self.weights = []
        for w in (layer.gate_up.detach(), layer.down.detach()):
            q = gemm.mx4_empty(w.shape[0] * w.shape[1], w.shape[2], w.device)
            self.weights.append((handle.mx4_quantise(w, q), w.shape[1]))

    def _product(self, x, i, offsets):
        weight, N = self.weights[i]
        xq = self.handle.mx4_quantise(x, gemm.mx4_empty(x.shape[0], x.shape[1], x.device))
        y = torch.empty((x.shape[0], N), dtype=x.dtype, device=x.device)
        return self.handle.run_mx4_grouped(xq, weight, offsets, y)

    @torch.no_grad()
    def __call__(self, x):
        prob, order, offsets = self.layer.route(x)
        gate, up = self._product(x[order // self.layer.top_k], 0, offsets).chunk(2, -1)
        y = self._product(F.silu(gate) * up, 1, offsets)
        return self.layer._combine(x, prob, order, y)


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--inner", type=int, default=1408)
    ap.add_argument("--experts", type=int, default=32)
    ap.add_argument("--top-k", type=int, default=4)
    ap.add_argument("--steps", type=int, default=5)
    a = ap.parse_args(argv)
    torch.manual_seed(0)
    layer = ExpertLayer(a.hidden, a.inner, a.experts, a.top_k)
    x = torch.randn(a.tokens, a.hidden, device="cuda").bfloat16()
    target = torch.randn(a.tokens, a.hidden, device="cuda") * 0.5
    losses = []
    opt = torch.optim.SGD(layer.parameters(), lr=0.1 * a.hidden)
    for _ in range(a.steps):
        opt.zero_grad()
        loss = (layer(x).float() - target).square().mean()
        loss.backward()
        opt.step()
        losses.append(loss.item())
    print("losses of the BF16 training steps:", " ".join(f"{v:.4f}" for v in losses))
    errors = {}
    with gemm.Gemm(0) as handle:
        served = ServedExpertLayer(layer, handle)
        for tokens in (a.tokens, 1):
            full = layer(x[:tokens]).detach().float()
            got = served(x[:tokens]).float()
            handle.sync_status()
            errors[tokens] = ((got - full).norm() / full.norm()).item()
            print(f"{tokens} tokens with 4-bit experts: {errors[tokens]:.3f} of the BF16 output's norm away "
                  f"({handle.last_path})")
    return losses, errors


if __name__ == "__main__":
    main()
