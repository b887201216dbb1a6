"""A routed feed-forward layer served with 8-bit integer matrices: a router by groups
of experts with a bias that balances their load, experts and one shared expert
with int8 codes and a scale for each channel, tokens quantised on the way in; and
the router's training through torch.autograd.

    python examples/moe_layer_i8.py [--tokens 2048] [--hidden 1024] [--ffn 512] [--experts 32] [--groups 8] [--top-k 4]

Nothing between the router and the layer's output goes through the host, so a
decoding step is captured in a HIP graph.
"""
from __future__ import annotations

import argparse
import sys
from pathlib import Path

import torch

sys.path.insert(0, str(Path(__file__).resolve().parent.parent))

import dense_block_scaled_amd as dbs  # noqa: E402


class RouterFunction(torch.autograd.Function):
    """weights, experts, offsets, rows, slots = router(logits, bias); the weights have a
    gradient with respect to the logits, the choice has none."""

    @staticmethod
    def forward(ctx, logits, bias, k, groups, kept, scale):
        r = dbs.moe_route_grouped(logits, k, bias, groups, kept, scale=scale)
        ctx.save_for_backward(logits, r.experts)
        ctx.scale = scale
        ctx.mark_non_differentiable(r.experts, r.offsets, r.rows, r.slots)
        return r.weights, r.experts, r.offsets, r.rows, r.slots

    @staticmethod
    def backward(ctx, dweights, *_):
        if torch.is_grad_enabled():                # (create_graph=True)
            raise RuntimeError("RouterFunction has no second derivatives: its gradient would be taken for a constant")
        logits, experts = ctx.saved_tensors
        d = dbs.moe_route_grouped_backward(logits, experts, dweights.contiguous(), scale=ctx.scale)
        return d, None, None, None, None, None


def quantised(w: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    """Codes and channel scales of matrices (..., N, K)."""
    q, s = dbs.quant_i8(w.reshape(-1, w.shape[-1]))
    return q.view(w.shape), s.view(w.shape[:-1])


class MoeLayerI8(torch.nn.Module):
    def __init__(self, hidden: int, ffn: int, experts: int, groups: int, k: int):
        super().__init__()
        self.k, self.groups, self.kept, self.scale = k, groups, max(1, groups // 2), 2.5
        self.router = torch.nn.Parameter(torch.randn(hidden, experts, device="cuda") * hidden ** -0.5)
        self.bias = torch.zeros(experts, device="cuda")

        def matrices(*shape):
            return quantised(torch.randn(*shape, device="cuda") * shape[-1] ** -0.5)

        self.q13, self.s13 = matrices(experts, 2 * ffn, hidden)
        self.q2, self.s2 = matrices(experts, hidden, ffn)
        self.shared13, self.shared2 = matrices(2 * ffn, hidden), matrices(hidden, ffn)

    def route(self, x: torch.Tensor) -> dbs.MoeRouting:
        w, experts, offsets, rows, slots = RouterFunction.apply(x.float() @ self.router, self.bias, self.k, self.groups,
                                                                self.kept, self.scale)
        return dbs.MoeRouting(experts, w, offsets, rows, slots)

    def rows(self, x: torch.Tensor, r: dbs.MoeRouting) -> torch.Tensor:
        """The experts' results in sorted order, (T k, hidden)."""
        qx, sx = dbs.quant_i8(x)
        a = dbs.gemm_moe_swiglu_i8(qx, sx, self.q13, self.s13, r.offsets, r.rows)
        qa, sa = dbs.quant_i8(a)
        return dbs.gemm_moe_i8(qa, sa, self.q2, self.s2, r.offsets)

    def shared(self, x: torch.Tensor) -> torch.Tensor:
        h = dbs.gemm_i8(*dbs.quant_i8(x), *self.shared13)
        return dbs.gemm_i8(*dbs.quant_i8(dbs.swiglu(h)), *self.shared2)

    @torch.no_grad()
    def forward(self, x: torch.Tensor) -> torch.Tensor:
        r = self.route(x)
        return dbs.moe_combine(self.rows(x, r), r.slots, r.weights) + self.shared(x)

    def router_loss(self, x: torch.Tensor, target: torch.Tensor) -> torch.Tensor:
        """What the router learns from with the matrices frozen: the distance of the
        weighted sums of the experts' rows from a target."""
        r = self.route(x)
        with torch.no_grad():
            y = self.rows(x, r).float()
        at = r.slots.long().clamp(min=0)
        out = (r.weights[..., None] * y[at] * (r.slots >= 0)[..., None]).sum(1)
        return (out - target).square().mean()

    @torch.no_grad()
    def balance(self, r: dbs.MoeRouting, step: float = 1e-3) -> None:
        """Experts with more than their share of the pairs become less likely to be
        chosen, whatever their weights."""
        load = r.offsets.diff().float()
        self.bias -= step * torch.sign(load - load.mean())


def reference(layer: MoeLayerI8, x: torch.Tensor) -> torch.Tensor:
    """The layer in plain operations on the same (dequantised) matrices, tokens not quantised."""
    silu = torch.nn.functional.silu
    x = x.float()
    s = torch.sigmoid((x @ layer.router).double())
    T, E = s.shape
    by = (s + layer.bias.double()).view(T, layer.groups, -1)
    group = by.topk(min(2, by.shape[2]), dim=2).values.sum(2)
    keep = torch.zeros_like(group).scatter_(1, group.topk(layer.kept, dim=1).indices, 1.0)
    e = torch.where(keep[..., None] > 0, by, -torch.inf).view(T, E).topk(layer.k, dim=1).indices
    w = s.gather(1, e)
    w = (w / w.sum(1, keepdim=True) * layer.scale).float()
    w13, w2 = layer.q13.float() * layer.s13[..., None], layer.q2.float() * layer.s2[..., None]
    out = torch.zeros_like(x)
    for i in range(E):
        t, j = torch.nonzero(e == i, as_tuple=True)
        if t.numel():
            g, u = (x[t] @ w13[i].t()).chunk(2, dim=1)
            out.index_add_(0, t, w[t, j, None] * ((silu(g) * u) @ w2[i].t()))
    (q1, s1), (q2, s2) = layer.shared13, layer.shared2
    g, u = (x @ (q1.float() * s1[:, None]).t()).chunk(2, dim=1)
    return out + (silu(g) * u) @ (q2.float() * s2[:, None]).t()


def relative(a: torch.Tensor, b: torch.Tensor) -> float:
    a, b = a.detach().double(), b.detach().double()
    return float((a - b).norm() / b.norm())


def run(tokens: int, hidden: int, ffn: int, experts: int, groups: int, k: int, seed: int = 0) -> dict:
    """A prompt, a captured decoding step and a step of the router; the relative
    distance of the results from the reference, whose tokens are not quantised."""
    torch.manual_seed(seed)
    layer = MoeLayerI8(hidden, ffn, experts, groups, k)
    x = torch.randn(tokens, hidden, device="cuda", dtype=torch.bfloat16)
    want = reference(layer, x)
    far = {"out": relative(layer(x), want)}

    # a decoding step of one token, captured once and replayed on new inputs
    token = torch.empty(1, hidden, device="cuda", dtype=torch.bfloat16)
    token.copy_(x[:1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(token)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        result = layer(token)
    for i in range(min(3, tokens)):
        token.copy_(x[i:i + 1])
        graph.replay()
        far[f"token {i}"] = relative(result, want[i:i + 1])

    layer.router_loss(x, torch.randn_like(want)).backward()
    far["router gradient, norm"] = float(layer.router.grad.norm())
    layer.balance(layer.route(x))
    return far


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--ffn", type=int, default=512)
    ap.add_argument("--experts", type=int, default=32)
    ap.add_argument("--groups", type=int, default=8)
    ap.add_argument("--top-k", type=int, default=4)
    a = ap.parse_args()
    for name, v in run(a.tokens, a.hidden, a.ffn, a.experts, a.groups, a.top_k).items():
        print(f"{name:22s} {v:.2e}", flush=True)


if __name__ == "__main__":
    main()
