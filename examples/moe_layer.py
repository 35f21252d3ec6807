"""One mixture-of-experts layer from tokens to tokens, forward and backward.

    logits = x . w_router
    ids, weights = the k experts of every token       (gmm_route)
    rows = x in the order of the experts              (gmm_sort_tokens, gmm_dispatch)
    h = act(rows . w_up[g] + b_up[g])                 (gmm_bf16_linear), or the gated
        silu(rows . w_gate[g]) * (rows . w_up[g])     (gmm_bf16_swiglu)
    y = h . w_down[g] + b_down[g]                     (gmm_bf16_linear)
    out = x + weights * y of every token's experts    (gmm_combine)

    python examples/moe_layer.py [--tokens 8192 --experts 32 --top-k 4 --k 2048 --n 512 --gated]

prints the time of a forward and of a backward pass.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import moe_grouped_gemm_gmm_amd as gmm  # noqa: E402


class MoeLayer:
    """Weights: w_router [K,E] bf16, w_up [E,K,N] (gated: [E,K,2N], gate columns first), w_down [E,N,K]; biases b_up
    [E,N] (not gated) and b_down [E,K].  One rank of an expert-parallel group holds the experts first .. first + G - 1."""

    def __init__(self, w_router, w_up, b_up, w_down, b_down, top_k, activation="gelu", gated=False, first=0, **route):
        self.w_router, self.w_up, self.b_up, self.w_down, self.b_down = w_router, w_up, b_up, w_down, b_down
        self.top_k, self.activation, self.gated, self.first, self.route = top_k, activation, gated, first, route

    def forward(self, x):
        """(out [T,K], what the backward pass needs)."""
        G, M = self.w_down.shape[0], x.shape[0] * self.top_k
        logits = x @ self.w_router
        ids, weights = gmm.gmm_route(logits, self.top_k, **self.route)
        gs, row_of, slot_of = gmm.gmm_sort_tokens(ids, G, first=self.first)
        rows = gmm.gmm_dispatch(x, row_of, slot_of)
        pre = torch.empty((M, self.w_up.shape[2]), dtype=torch.bfloat16, device=x.device)
        if self.gated:
            h = gmm.gmm_bf16_swiglu(rows, self.w_up, gs, gu=pre)
        else:
            h = gmm.gmm_bf16_linear(rows, self.w_up, gs, bias=self.b_up, activation=self.activation, pre=pre)
        y = gmm.gmm_bf16_linear(h, self.w_down, gs, bias=self.b_down)
        out = gmm.gmm_combine(y, row_of, weights=weights, residual=x)
        return out, (x, logits, ids, weights, gs, row_of, slot_of, rows, pre, h, y)

    def backward(self, dout, kept):
        """Gradients of x and of the weights, in the constructor's order."""
        x, logits, ids, weights, gs, row_of, slot_of, rows, pre, h, y = kept
        dy, dweights = gmm.gmm_combine_bwd(dout, y, row_of, slot_of, weights)
        dh, dw_down, db_down = gmm.gmm_bf16_linear_bwd(dy, self.w_down, gs, lhs=h)
        if self.gated:
            drows, dw_up = gmm.gmm_bf16_swiglu_bwd(dh, self.w_up, gs, lhs=rows, gu=pre)
            db_up = None
        else:
            drows, dw_up, db_up = gmm.gmm_bf16_linear_bwd(dh, self.w_up, gs, lhs=rows, pre=pre, activation=self.activation)
        how = {k: v for k, v in self.route.items() if k != "bias"}   # the bias chooses; nothing flows through the choice
        dlogits = gmm.gmm_route_bwd(dweights, logits, ids, **how)
        dx = gmm.gmm_combine(drows, row_of, residual=dout) + dlogits @ self.w_router.t()
        return dx, x.t() @ dlogits, dw_up, db_up, dw_down, db_down


def make(tokens, experts, top_k, k, n, gated=False, seed=0, device="cuda:0", **how):
    """A layer with random weights, an input and an output gradient."""
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    r = lambda shape, s: torch.randn(shape, generator=gen, device=device, dtype=torch.bfloat16).mul_(s)
    layer = MoeLayer(r((k, experts), k ** -0.5), r((experts, k, n * (2 if gated else 1)), k ** -0.5),
                     None if gated else r((experts, n), 0.1), r((experts, n, k), n ** -0.5), r((experts, k), 0.1), top_k,
                     gated=gated, **how)
    return layer, r((tokens, k), 1.0), r((tokens, k), 0.1)


def run(tokens=8192, experts=32, top_k=4, k=2048, n=512, gated=False, steps=10, **how):
    """(milliseconds of a forward pass, of a backward pass, out, gradients)."""
    layer, x, dout = make(tokens, experts, top_k, k, n, gated, **how)
    for _ in range(3):
        out, kept = layer.forward(x)
        grads = layer.backward(dout, kept)
    t = [torch.cuda.Event(enable_timing=True) for _ in range(3)]
    t[0].record()
    for _ in range(steps):
        out, kept = layer.forward(x)
    t[1].record()
    for _ in range(steps):
        grads = layer.backward(dout, kept)
    t[2].record()
    torch.cuda.synchronize()
    return t[0].elapsed_time(t[1]) / steps, t[1].elapsed_time(t[2]) / steps, out, grads


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("tokens", 8192), ("experts", 32), ("top-k", 4), ("k", 2048), ("n", 512)):
        p.add_argument("--" + name, type=int, default=default)
    p.add_argument("--gated", action="store_true")
    a = p.parse_args()
    fwd, bwd, _, _ = run(a.tokens, a.experts, a.top_k, a.k, a.n, a.gated)
    print("forward %.3f ms, backward %.3f ms" % (fwd, bwd))


if __name__ == "__main__":
    main()
