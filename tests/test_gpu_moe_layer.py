"""GPU: the calls of include/gmm_moe.h together, as a layer uses them: forward and
backward against float64 on the CPU, under HIP graphs, on several streams, and
over expert-parallel ranks.

Bounds.  Every tensor handed from one call to the next is bf16 (2^-8 of it), so a
value is compared by norm: each of the at most eight roundings on a path moves
it by at most 2^-8 of its norm, and fp32 sums add little beside them."""
import os
import sys

import pytest
import torch

import moe_grouped_gemm_gmm_amd as gmm

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import moe_layer  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
STEP = 2.0 ** -8


def reference(layer, x, dout, logits, ids):
    """out and gradients in float64 by autograd, with the layer's logits and choices."""
    p = {n: getattr(layer, n) for n in ("w_router", "w_up", "b_up", "w_down", "b_down")}
    p = {n: None if v is None else v.double().cpu().requires_grad_() for n, v in p.items()}
    xd = x.double().cpu().requires_grad_()
    how = {"score": "softmax", "normalize": True, "scale": 1.0, **{k: v for k, v in layer.route.items() if k != "bias"}}
    l = xd @ p["w_router"]
    l = l + (logits.double().cpu() - l).detach()          # the rounded logits, the gradient of the exact ones
    s = torch.softmax(l, 1) if how["score"] == "softmax" else torch.sigmoid(l)
    ids = ids.long().cpu()
    w = s.gather(1, ids)
    if how["normalize"]:
        w = w / w.sum(1, keepdim=True)
    w = w * how["scale"]
    G, first = layer.w_down.shape[0], layer.first
    out = xd
    for g in range(G):
        t, j = torch.nonzero(ids == first + g, as_tuple=True)
        z = xd[t] @ p["w_up"][g]
        if layer.gated:
            n = z.shape[1] // 2
            h = torch.nn.functional.silu(z[:, :n]) * z[:, n:]
        else:
            h = torch.nn.functional.gelu(z + p["b_up"][g])
        y = h @ p["w_down"][g] + p["b_down"][g]
        out = out.index_add(0, t, w[t, j][:, None] * y)
    (out * dout.double().cpu()).sum().backward()
    return out.detach(), [xd.grad] + [None if p[n] is None else p[n].grad
                                      for n in ("w_router", "w_up", "b_up", "w_down", "b_down")]


def near(got, want, roundings=8):
    got = got.double().cpu()
    assert torch.isfinite(got).all()
    assert (got - want).norm() <= roundings * STEP * want.norm(), ((got - want).norm() / want.norm()).item()


CASES = [dict(tokens=1, experts=8, top_k=2, k=128, n=64), dict(tokens=203, experts=12, top_k=3, k=192, n=128),
         dict(tokens=203, experts=12, top_k=3, k=192, n=128, gated=True), dict(tokens=600, experts=5, top_k=5, k=256, n=320)]
HOW = [dict(), dict(normalize=False), dict(score="sigmoid", scale=2.5), dict(score="sigmoid", normalize=False)]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("how", HOW)
def test_layer(case, how):
    layer, x, dout = moe_layer.make(seed=3, **case, **how)
    if how.get("score") == "sigmoid":
        layer.route["bias"] = torch.randn(case["experts"], generator=torch.Generator().manual_seed(1)).mul(0.1).to(DEV)
    out, kept = layer.forward(x)
    grads = layer.backward(dout, kept)
    assert int(kept[4].sum()) == case["tokens"] * case["top_k"]
    want, wgrads = reference(layer, x, dout, kept[1], kept[2])
    near(out, want)
    for i, (g, r) in enumerate(zip(grads, wgrads)):
        if r is not None and r.norm() > 1e-6 * dout.double().norm().cpu():   # one expert of one: its weight is always 1
            # the router's gradient goes through dweights, differences of sums of magnitude of the whole dot products
            near(g, r, 8 if i > 1 else 24)


def test_expert_parallel_ranks_add_up():
    """Each rank sorts and computes its own experts; the tokens' sums over ranks are the whole layer's."""
    layer, x, dout = moe_layer.make(tokens=300, experts=12, top_k=4, k=128, n=64, seed=5)
    out, kept = layer.forward(x)
    ids, weights = kept[2], kept[3]
    total = x.double()
    for first in (0, 5, 9):
        G = {0: 5, 5: 4, 9: 3}[first]
        rows = int(((ids >= first) & (ids < first + G)).sum()) + 7            # a buffer of its own size
        gs, row_of, slot_of = gmm.gmm_sort_tokens(ids, G, first=first, rows=rows)
        e = slice(first, first + G)
        h = gmm.gmm_bf16_linear(gmm.gmm_dispatch(x, row_of, slot_of), layer.w_up[e].contiguous(), gs,
                                bias=layer.b_up[e].contiguous(), activation="gelu")
        y = gmm.gmm_bf16_linear(h, layer.w_down[e].contiguous(), gs, bias=layer.b_down[e].contiguous())
        total = total + gmm.gmm_combine(y, row_of, weights=weights, out_dtype=F32).double()
    # the whole layer's out is rounded to bf16 once
    assert ((out.double() - total).abs() <= STEP * total.abs() + 1e-5).all()


def steps():
    """A step of everything, on buffers that stay; (function, its outputs)."""
    T, E, k, K, N = 700, 24, 3, 192, 320
    layer, x, dout = moe_layer.make(T, E, k, K, N, seed=9)
    logits = (x @ layer.w_router).float()
    bias = torch.randn(E, device=DEV) * 0.05
    made = {}

    def run():
        ids, w = gmm.gmm_route(logits, k, bias=bias, score="sigmoid", scale=2.0)
        gs, row_of, slot_of = gmm.gmm_sort_tokens(ids, E, rows=T * k - 50)
        big = gmm.gmm_sort_tokens(ids.repeat(3, 1), E)                          # more than one workgroup's
        rows = gmm.gmm_dispatch(x, row_of, slot_of)
        pre = torch.empty((rows.shape[0], N), dtype=BF, device=DEV)
        h = gmm.gmm_bf16_linear(rows, layer.w_up, gs, bias=layer.b_up, activation="gelu", pre=pre)
        y = gmm.gmm_bf16_linear(h, layer.w_down, gs, bias=layer.b_down)
        out = gmm.gmm_combine(y, row_of, weights=w, residual=x)
        dy, dw = gmm.gmm_combine_bwd(dout, y, row_of, slot_of, w)
        dh, dwd, dbd = gmm.gmm_bf16_linear_bwd(dy, layer.w_down, gs, lhs=h)
        drows, dwu, dbu = gmm.gmm_bf16_linear_bwd(dh, layer.w_up, gs, lhs=rows, pre=pre, activation="gelu")
        dx = gmm.gmm_combine(drows, row_of, residual=dout)
        dl = gmm.gmm_route_bwd(dw, logits, ids, score="sigmoid", scale=2.0)
        made["out"] = (ids, w, gs, row_of, slot_of) + big + (rows, pre, h, y, out, dy, dw, dh, dwd, dbd, drows, dwu, dbu, dx, dl)

    return run, made, x


def test_graph_replays_match_eager():
    run, made, x = steps()
    run()
    torch.cuda.synchronize()
    eager = [t.clone() for t in made["out"]]
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        run()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            run()
    torch.cuda.synchronize()
    got = made["out"]
    for rep in range(4):
        for t in got:
            t.zero_()                                     # eager work between replays
        junk = (torch.randn(1 << 20, device=DEV) * 3).sum()
        run()                                             # and the same calls, eagerly
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.isfinite(junk)
        for i, (a, b) in enumerate(zip(got, eager)):
            assert torch.equal(a, b), (rep, i)


def test_two_graphs_at_once():
    """Two captured steps replayed together on two streams: neither's workspaces are the other's."""
    a, b = steps(), steps()
    graphs = []
    for run, made, _ in (a, b):
        run()
        torch.cuda.synchronize()
        want = [t.clone() for t in made["out"]]
        s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.stream(s):
            run()
            torch.cuda.synchronize()
            with torch.cuda.graph(g, stream=s):
                run()
        torch.cuda.synchronize()
        graphs.append((s, g, made["out"], want))
    for rep in range(5):
        for _, _, got, _ in graphs:
            for t in got:
                t.zero_()
        torch.cuda.synchronize()
        for s, g, _, _ in graphs:
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for _, _, got, want in graphs:
            assert all(torch.equal(u, v) for u, v in zip(got, want)), rep


def test_new_tokens_in_a_captured_step():
    """A replay reads what its inputs hold then: another routing, other sizes of the groups."""
    T, E, k, K, N = 256, 16, 2, 128, 128
    layer, x, _ = moe_layer.make(T, E, k, K, N, seed=1)
    logits = torch.randn(T, E, device=DEV)

    def run():
        ids, w = gmm.gmm_route(logits, k)
        gs, row_of, slot_of = gmm.gmm_sort_tokens(ids, E)
        h = gmm.gmm_bf16_linear(gmm.gmm_dispatch(x, row_of, slot_of), layer.w_up, gs, activation="silu")
        return ids, gs, gmm.gmm_combine(gmm.gmm_bf16_linear(h, layer.w_down, gs), row_of, weights=w)

    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        run()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            got = run()
    torch.cuda.synchronize()
    for seed in range(4):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        logits.copy_(torch.randn(T, E, generator=g, device=DEV) * (1 + 3 * seed))
        logits[:, seed * 3:seed * 3 + 2] = float("-inf")
        x.copy_(torch.randn(T, K, generator=g, device=DEV))
        want = run()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_in_place():
    """The outputs that may be one of the inputs."""
    T, E, k, K = 300, 20, 4, 136
    logits = torch.randn(T, E, device=DEV)
    ids, w = gmm.gmm_route(logits, k)
    dw = torch.randn(T, k, device=DEV)
    for dt in (F32, BF):
        for normalize in (True, False):
            l = logits.to(dt)
            want = gmm.gmm_route_bwd(dw, l, ids, normalize=normalize)
            assert gmm.gmm_route_bwd(dw, l, ids, normalize=normalize, out=l) is l and torch.equal(l, want)
        _, row_of, slot_of = gmm.gmm_sort_tokens(ids, E, rows=T * k + 20)
        y, d = torch.randn(T * k + 20, K, device=DEV).to(dt), torch.randn(T, K, device=DEV).to(dt)
        dy, dweights = gmm.gmm_combine_bwd(d, y, row_of, slot_of, w)
        again = gmm.gmm_combine_bwd(d, y, row_of, slot_of, w, dy=y)
        assert again[0] is y and torch.equal(y, dy) and torch.equal(again[1], dweights)


def test_example_runs():
    for gated in (False, True):
        fwd, bwd, out, grads = moe_layer.run(tokens=512, experts=8, top_k=2, k=256, n=128, gated=gated, steps=2)
        assert fwd > 0 and bwd > 0 and torch.isfinite(out.float()).all()
        assert all(g is None or torch.isfinite(g.float()).all() for g in grads)
