"""A routed feed-forward layer on the mixture-of-experts operators: a training
step through torch.autograd and a decoding step captured in a HIP graph.

    python examples/moe_layer.py [--tokens 2048] [--hidden 1024] [--ffn 512] [--experts 32] [--top-k 4]

Training keeps the gate's inputs and runs every operator in both directions;
decoding uses the gate fused into the first product.  Nothing between the
router and the layer's output goes through the host.
"""
from __future__ import annotations

import argparse
import sys
from pathlib import Path

import torch

sys.path.insert(0, str(Path(__file__).resolve().parent.parent))

import dense_block_scaled_amd as dbs  # noqa: E402


class MoeFunction(torch.autograd.Function):
    """out = layer(x, logits, w13, w2); gradients of those of the four that need
    one (first ones: the operators have no second derivatives)."""

    @staticmethod
    def forward(ctx, x, logits, w13, w2, k):
        r = dbs.moe_route(logits, k)
        h = dbs.gemm_moe_bf16(x, w13, r.offsets, r.rows)
        a = dbs.swiglu(h)
        y = dbs.gemm_moe_bf16(a, w2, r.offsets)
        ctx.save_for_backward(x, logits, w13, w2, h, a, y, *r)
        return dbs.moe_combine(y, r.slots, r.weights)

    @staticmethod
    def backward(ctx, dout):
        if torch.is_grad_enabled():                # (create_graph=True)
            raise RuntimeError("MoeFunction has no second derivatives: its gradients would be taken for constants")
        x, logits, w13, w2, h, a, y, *r = ctx.saved_tensors
        need_x, need_logits, need_w13, need_w2, _ = ctx.needs_input_grad
        r = dbs.MoeRouting(*r)
        dx = dlogits = dw13 = dw2 = None
        dy, dweights = dbs.moe_combine_backward(dout.contiguous(), y, r.slots, r.weights, r.offsets)
        if need_w2:
            dw2 = dbs.gemm_moe_dw_bf16(dy, a, r.offsets)
        if need_x or need_w13:
            da = dbs.gemm_moe_bf16(dy, w2, r.offsets, lw=dbs.MN_MAJOR)    # w2 (E, H, F) as K x N
            dh = dbs.swiglu_backward(da, h)
        if need_w13:
            dw13 = dbs.gemm_moe_dw_bf16(dh, x, r.offsets, r.rows)
        if need_x:
            dxs = dbs.gemm_moe_bf16(dh, w13, r.offsets, lw=dbs.MN_MAJOR)
            dx = dbs.moe_combine(dxs, r.slots)                            # a token's rows, summed
        if need_logits:
            dlogits = dbs.moe_route_backward(logits, r.experts, dweights)
        return dx, dlogits, dw13, dw2, None


class MoeLayer(torch.nn.Module):
    def __init__(self, hidden: int, ffn: int, experts: int, k: int):
        super().__init__()
        self.k = k
        bf = dict(dtype=torch.bfloat16, device="cuda")
        self.router = torch.nn.Parameter(torch.randn(hidden, experts, device="cuda") * hidden ** -0.5)
        self.w13 = torch.nn.Parameter(torch.randn(experts, 2 * ffn, hidden, **bf) * hidden ** -0.5)
        self.w2 = torch.nn.Parameter(torch.randn(experts, hidden, ffn, **bf) * ffn ** -0.5)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        return MoeFunction.apply(x, x.float() @ self.router, self.w13, self.w2, self.k)

    @torch.no_grad()
    def decode(self, x: torch.Tensor) -> torch.Tensor:
        """The layer for a few tokens: router, gated first product, second
        product, sum -- four kernels of the library."""
        r = dbs.moe_route(x.float() @ self.router, self.k)
        a = dbs.gemm_moe_swiglu_bf16(x, self.w13, r.offsets, r.rows)
        return dbs.moe_combine(dbs.gemm_moe_bf16(a, self.w2, r.offsets), r.slots, r.weights)


def reference(layer: MoeLayer, x: torch.Tensor, router, w13, w2) -> torch.Tensor:
    """The layer in plain operations, expert by expert."""
    logits = x @ router
    p, e = logits.topk(layer.k, dim=1)
    p = torch.softmax(p, dim=1)
    out = torch.zeros_like(x)
    for i in range(w13.shape[0]):
        t, j = torch.nonzero(e == i, as_tuple=True)
        if t.numel():
            g, u = (x[t] @ w13[i].t()).chunk(2, dim=1)
            out = out.index_add(0, t, p[t, j, None] * ((torch.nn.functional.silu(g) * u) @ w2[i].t()))
    return out


def relative(a: torch.Tensor, b: torch.Tensor) -> float:
    a, b = a.detach().double(), b.detach().double()
    return float((a - b).norm() / b.norm())


def run(tokens: int, hidden: int, ffn: int, experts: int, k: int, seed: int = 0) -> dict:
    """One training step and one captured decoding step; the relative
    distance of every result from the reference in 32 bits."""
    torch.manual_seed(seed)
    layer = MoeLayer(hidden, ffn, experts, k)
    x = torch.randn(tokens, hidden, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    out = layer(x)
    g = torch.randn_like(out)
    out.backward(g)

    ref = [t.detach().float().requires_grad_() for t in (x, layer.router, layer.w13, layer.w2)]
    want = reference(layer, *ref)
    want.backward(g.float())
    far = {"out": relative(out, want)}
    for name, got, r in zip(("dx", "drouter", "dw13", "dw2"), (x, layer.router, layer.w13, layer.w2), ref):
        far[name] = relative(got.grad, r.grad)

    # a decoding step of one token, captured once and replayed on new inputs
    token = torch.empty(1, hidden, device="cuda", dtype=torch.bfloat16)
    token.copy_(x[:1].detach())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.decode(token)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        result = layer.decode(token)
    for i in range(3):
        token.copy_(x[i:i + 1].detach())
        graph.replay()
        far[f"token {i}"] = relative(result, want[i:i + 1])
    return far


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--ffn", type=int, default=512)
    ap.add_argument("--experts", type=int, default=32)
    ap.add_argument("--top-k", type=int, default=4)
    a = ap.parse_args()
    for name, v in run(a.tokens, a.hidden, a.ffn, a.experts, a.top_k).items():
        print(f"{name:10s} relative distance {v:.2e}", flush=True)


if __name__ == "__main__":
    main()
