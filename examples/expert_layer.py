"""One training step of a mixture-of-experts layer, rows already sorted by expert.

    P = x . Wgu[g],  h = silu(gate) * up,  y = h . Wd[g]          forward
    dh = dy . Wd^T,  dWd = h^T dy,  dx, dWgu from dh              backward

What the backward pass needs is kept either in bfloat16 (x, P and h: K + 3N
values a row, 2 bytes each) or as 8-bit checkpoints of x and P with h
recomputed from P (K + 2N values a row, 1.03 bytes each).

    python examples/expert_layer.py [--rows 8192 --experts 32 --k 2048 --n 512]

prints the bytes kept, the time of a step and how far the gradients of the
two forms are apart.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import moe_grouped_gemm_gmm_amd as gmm  # noqa: E402


class ExpertLayer:
    """Weights of G gated experts: w_gate_up [G,K,2N] (gate columns first), w_down [G,N,K], bf16."""

    def __init__(self, w_gate_up: torch.Tensor, w_down: torch.Tensor, eight_bit: bool):
        self.w_gate_up, self.w_down, self.eight_bit = w_gate_up, w_down, eight_bit

    def forward(self, x: torch.Tensor, group_sizes: torch.Tensor):
        """(y [M,K], what the backward pass needs)."""
        M, N2 = x.shape[0], self.w_gate_up.shape[2]
        if self.eight_bit:
            x_q, x_s = gmm.gmm_quantize_mx8(x)
            gu_q = torch.empty((M, N2), dtype=torch.uint8, device=x.device)
            gu_s = torch.empty((M, N2 // 32), dtype=torch.uint8, device=x.device)
            h = gmm.gmm_bf16_swiglu(x, self.w_gate_up, group_sizes, gu_q=gu_q, gu_scale=gu_s)
            kept = dict(lhs_q=x_q, lhs_scale=x_s, gu_q=gu_q, gu_scale=gu_s)
        else:
            gu = torch.empty((M, N2), dtype=torch.bfloat16, device=x.device)
            h = gmm.gmm_bf16_swiglu(x, self.w_gate_up, group_sizes, gu=gu)
            kept = dict(lhs=x, gu=gu, h=h)
        return gmm.gmm_bf16_fwd(h, self.w_down, group_sizes), kept

    def backward(self, dy: torch.Tensor, group_sizes: torch.Tensor, kept: dict):
        """(dx, dw_gate_up, dw_down) from dy [M,K]."""
        kept = dict(kept)
        h = kept.pop("h", None)
        again = torch.empty((dy.shape[0], self.w_down.shape[1]), dtype=torch.bfloat16, device=dy.device) \
            if h is None else None
        dh = gmm.gmm_bf16_dx(dy, self.w_down, group_sizes)
        dx, dw_gate_up = gmm.gmm_bf16_swiglu_bwd(dh, self.w_gate_up, group_sizes, h=again, **kept)
        return dx, dw_gate_up, gmm.tgmm_bf16(again if h is None else h, dy, group_sizes)


def bytes_kept(kept: dict) -> int:
    return sum(t.numel() * t.element_size() for t in kept.values())


def run(rows=8192, experts=32, k=2048, n=512, seed=0, device="cuda:0"):
    """The same step with both kinds of kept activations: (bytes kept, gradients) of each."""
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    r = lambda shape, s: torch.randn(shape, generator=gen, device=device, dtype=torch.bfloat16).mul_(s)
    sizes = torch.bincount(torch.randint(0, experts, (rows,), generator=gen, device=device), minlength=experts)
    gs = sizes.to(torch.int32)
    x, dy = r((rows, k), 1.0), r((rows, k), 0.1)
    w_gate_up, w_down = r((experts, k, 2 * n), k ** -0.5), r((experts, n, k), n ** -0.5)
    out = []
    for eight_bit in (False, True):
        layer = ExpertLayer(w_gate_up, w_down, eight_bit)

        def step():
            y, kept = layer.forward(x, gs)
            return y, kept, layer.backward(dy, gs, kept)

        for _ in range(3):
            y, kept, grads = step()
        t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        t0.record()
        for _ in range(10):
            y, kept, grads = step()
        t1.record()
        torch.cuda.synchronize()
        out.append(dict(kept=bytes_kept(kept), ms=t0.elapsed_time(t1) / 10, y=y, grads=grads))
    return out


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("rows", 8192), ("experts", 32), ("k", 2048), ("n", 512)):
        p.add_argument("--" + name, type=int, default=default)
    a = p.parse_args()
    plain, small = run(a.rows, a.experts, a.k, a.n)
    for name, o in (("bfloat16", plain), ("8-bit checkpoints", small)):
        print("%-18s %7.1f MB kept, %.3f ms a step" % (name, o["kept"] / 1e6, o["ms"]))
    for name, u, v in zip(("dx", "dw_gate_up", "dw_down"), plain["grads"], small["grads"]):
        print("%-10s the two differ by %.4f of its norm"
              % (name, ((u.float() - v.float()).norm() / u.float().norm()).item()))


if __name__ == "__main__":
    main()
