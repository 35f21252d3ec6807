"""What stands around the experts' products in one mixture-of-experts layer, as a user's program calls it.

Three things that belong together, each with its gradient:

* the router: from a token's scores of all experts, the k experts that it goes
  to and their weights;
* tokens sorted by expert and back: the sorted order of the rows, the rows
  moved into it, and every token's k results added with the router's weights;
* the grouped product with its epilogue, for experts that are not gated or
  have biases: pre = x . w[g] + b[g], out = act(pre) + residual.

Kinds of cases (case["op"]):
  route     ids and weights of T tokens, and with case["grad"] the gradient of
            the scores; score "softmax" or "sigmoid"; "bias": the choice is by
            score + bias (the weights are not); "masked": some experts are off
            (-inf) and a padding token has none left
  plan      the sorted order alone: group sizes, row of every slot, slot of
            every row (a slot is one of a token's k choices)
  move      the order, the rows moved into it, and a layer's results brought
            back: weights applied, residual added
  back      the gradient of that: of the results, the weights and the tokens
  linear    the grouped product with its epilogue; "pre": the sums are kept for
            the backward pass
  linear_bwd  its gradient: dx, dw, db
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one token of a 256-expert model, scored by a sigmoid with a balancing bias, top 8
        dict(name="route_one_token", op="route", T=1, E=256, k=8, dt="f32", score="sigmoid", bias=True,
             normalize=True, scale=2.5, masked=False, grad=False),
        # a ragged batch of a smaller model with two experts switched off and a padding token
        dict(name="route_odd", op="route", T=1777, E=60, k=6, dt="bf16", score="softmax", bias=False,
             normalize=True, scale=1.0, masked=True, grad=True),
        # the production batch's tokens, choice and gradient through the whole softmax
        dict(name="route_production", op="route", T=65536, E=256, k=8, dt="f32", score="softmax", bias=False,
             normalize=False, scale=1.0, masked=False, grad=True),
        # one token sent to eight of 256 experts and back
        dict(name="move_one_token", op="move", T=1, k=8, E=256, ranks=1, K=2048, dt="bf16", pad=0, zipf=False),
        # one of four expert-parallel ranks, whose buffer holds half of all slots; fp32 rows, padding tokens
        dict(name="move_rank_odd", op="move", T=1777, k=6, E=52, ranks=4, K=1088, dt="f32", pad=41, zipf=False),
        # the production batch: 65536 rows of 2048
        dict(name="move_production", op="move", T=8192, k=8, E=256, ranks=1, K=2048, dt="bf16", pad=0, zipf=True),
        # its gradient
        dict(name="back_production", op="back", T=8192, k=8, E=256, ranks=1, K=2048, dt="bf16", pad=0, zipf=True),
        # the order of eight such batches at once
        dict(name="plan_large", op="plan", T=65536, k=8, E=256, ranks=1, pad=0, zipf=True),
        # one token's eight experts: the down projection with a bias
        dict(name="linear_one_token", op="linear", M=8, G=256, K=512, N=2048, tail=0, route="one", act="none",
             bias=True, residual=False, pre=False, rseed=3),
        # odd widths, empty experts, unused rows; what the backward pass needs is kept
        dict(name="linear_odd", op="linear", M=1777, G=13, K=1088, N=704, tail=41, route="holes", act="silu",
             bias=True, residual=True, pre=True, rseed=11),
        # the production batch's down projection: 256 experts, skewed routing, bias and residual
        dict(name="linear_production", op="linear", M=65536, G=256, K=512, N=2048, tail=0, route="zipf", act="none",
             bias=True, residual=True, pre=False, rseed=31),
        # the expert-parallel shard's backward pass through GELU
        dict(name="linear_bwd_shard", op="linear_bwd", M=8192, G=32, K=2048, N=512, tail=0, route="uniform",
             act="gelu", rseed=17),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route", "plan", "move", "back", "linear", "linear", "linear_bwd"])
    if op == "route":
        while True:
            T, E = _log_int(rng, 1, 65536), _log_int(rng, 2, 512)
            if T * E <= 65536 * 256:
                break
        return dict(op=op, T=T, E=E, k=rng.randint(1, min(E, 16)), dt=rng.choice(["bf16", "f32"]),
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5,
                    normalize=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]), masked=rng.random() < 0.3,
                    grad=rng.random() < 0.6)
    if op in ("plan", "move", "back"):
        while True:
            T, E = _log_int(rng, 1, 65536), _log_int(rng, 2, 512)
            c = dict(op=op, T=T, k=rng.randint(1, min(E, 12)), E=E, ranks=rng.choice([1, 1, 2, 4]),
                     zipf=rng.random() < 0.5)
            if E % c["ranks"] or T * c["k"] > (524288 if op == "plan" else 65536):
                continue
            c["pad"] = rng.choice([0, rng.randrange(0, max(1, T // 8))])
            if op != "plan":
                c.update(K=8 * _log_int(rng, 8, 1024), dt=rng.choice(["bf16", "f32"]))
                if T * c["k"] * c["K"] * (2 if c["dt"] == "f32" else 1) > 65536 * 2048:
                    continue
            return c
    while True:
        c = dict(op=op, M=_log_int(rng, 1, 65536), G=_log_int(rng, 1, 256), K=64 * _log_int(rng, 1, 64),
                 N=64 * _log_int(rng, 1, 64), route=rng.choice(["uniform", "zipf", "holes", "one"]),
                 act=rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"]), rseed=rng.randrange(1 << 30))
        c["tail"] = rng.choice([0, rng.randrange(0, max(1, c["M"] // 4))])
        if op == "linear":
            c.update(bias=rng.random() < 0.7, residual=rng.random() < 0.5, pre=rng.random() < 0.5)
        products = 1 if op == "linear" else 2
        if products * c["M"] * c["K"] * c["N"] <= 65536 * 2048 * 512 and c["G"] * c["K"] * c["N"] <= 256 * 2048 * 512 \
                and c["M"] * max(c["K"], c["N"]) <= 65536 * 2048:
            return c


def sizes(case):
    """Rows of each expert of a grouped product: a property of the case (its routing)."""
    r = np.random.default_rng([case["rseed"], 101])
    M, G = case["M"] - case["tail"], case["G"]
    if case["route"] == "one" and M <= G:      # one row each for M distinct experts
        s = np.zeros(G, dtype=np.int64)
        s[r.choice(G, size=M, replace=False)] = 1
        return s
    p = np.ones(G)
    if case["route"] == "zipf":
        p = 1.0 / np.arange(1, G + 1)
        r.shuffle(p)
    elif case["route"] == "holes":             # about a third of the experts get nothing
        p = (r.random(G) > 0.35).astype(float)
        p[int(r.integers(G))] = 1.0
    return r.multinomial(M, p / p.sum()).astype(np.int64)


def local(case):
    """(first expert, experts, rows of the sorted buffer) of the rank whose order is made: the last one.  A rank's
    buffer has room for twice its even share."""
    E, n, slots = case["E"], case["ranks"], case["T"] * case["k"]
    return E - E // n, E // n, slots if n == 1 else min(slots, -(-2 * slots // n))


# ----------------------------------------------------------------- inputs --

def _normal(gen, shape, scale=1.0, dt=torch.bfloat16):
    return torch.randn(shape, generator=gen, device=DEV, dtype=dt).mul_(scale)


def _activations(gen, M, K, dt=torch.bfloat16):
    """Hidden states: unit normals with a few channels that run 8 times larger."""
    x = _normal(gen, (M, K), 1.0, dt)
    hot = torch.randint(0, K, (max(1, K // 256),), generator=gen, device=DEV)
    x[:, hot] *= 8.0
    return x


def _choices(case, gen):
    """Every token's k distinct experts (Gumbel noise on the experts' log popularity); padding tokens have none."""
    T, E, k = case["T"], case["E"], case["k"]
    pop = torch.zeros(E, device=DEV)
    if case["zipf"]:
        pop = -torch.log(1.0 + torch.randperm(E, generator=gen, device=DEV).float())
    u = torch.rand((T, E), generator=gen, device=DEV).clamp_(1e-7, 1 - 1e-7)
    ids = (pop - torch.log(-torch.log(u))).topk(k, dim=1).indices.to(torch.int32)
    if case["pad"]:
        ids[T - case["pad"]:] = -1
    return ids


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed) * 7919 + 29)
    op = case["op"]
    st = dict(case=case, op=op)
    if op == "route":
        T, E, dt = case["T"], case["E"], TYPES[case["dt"]]
        logits = (_normal(gen, (T, E), 1.2, torch.float32) + _normal(gen, (E,), 0.5, torch.float32)).to(dt)
        if case["masked"]:
            off = torch.randperm(E, generator=gen, device=DEV)[:E // 30 + 1]
            logits[:, off] = float("-inf")
            logits[T // 2] = float("-inf")     # a padding token
        st["logits"] = logits
        st["bias"] = _normal(gen, (E,), 0.05, torch.float32) if case["bias"] else None
        if case["grad"]:
            st["dweights"] = _normal(gen, (T, case["k"]), 1.0, torch.float32)
        return st
    if op in ("plan", "move", "back"):
        T, k = case["T"], case["k"]
        st["ids"] = _choices(case, gen)
        st["first"], st["G"], st["rows"] = local(case)
        if op == "plan":
            return st
        K, dt = case["K"], TYPES[case["dt"]]
        st["weights"] = torch.rand((T, k), generator=gen, device=DEV).add_(0.1).div_(k)
        gs, row_of, slot_of = _plain_order(st)
        used = int(gs.sum())
        st["y"] = _normal(gen, (st["rows"], K), 1.0, dt)
        st["y"][used:] = float("nan")          # rows of the buffer that no slot owns
        if op == "move":
            st["x"] = _activations(gen, T, K, dt)
            st["residual"] = _activations(gen, T, K, dt)
            return st
        st.update(row_of=row_of, slot_of=slot_of, dout=_normal(gen, (T, K), 0.25, dt),
                  drows=_normal(gen, (st["rows"], K), 0.25, dt))
        st["drows"][used:] = float("nan")
        return st
    M, G, K, N = case["M"], case["G"], case["K"], case["N"]
    s = sizes(case)
    used = int(s.sum())
    st.update(sizes=[int(v) for v in s], gs=torch.tensor(s, dtype=torch.int32, device=DEV))
    st["x"] = _activations(gen, M, K)
    st["x"][used:] = float("nan")              # rows of the buffer that no expert owns
    st["w"] = _normal(gen, (G, K, N), K ** -0.5)
    if op == "linear":
        st["bias"] = _normal(gen, (G, N), 0.5) if case["bias"] else None
        st["residual"] = _normal(gen, (M, N)) if case["residual"] else None
        if case["residual"]:
            st["residual"][used:] = float("nan")
        return st
    st["dout"] = _normal(gen, (M, N), 0.25)
    st["dout"][used:] = float("nan")
    st["pre"] = None
    if case["act"] != "none":
        st["pre"] = _normal(gen, (M, N), 1.2)
        st["pre"][used:] = float("nan")
    return st


# ------------------------------------------------------------ plain forms --

def _plain_route(st):
    c, logits = st["case"], st["logits"]
    k = c["k"]
    l = logits.float()
    on = l > float("-inf")
    p = torch.softmax(torch.where(on, l, torch.full_like(l, -1e30)), 1) if c["score"] == "softmax" else torch.sigmoid(l)
    p = torch.where(on, p, torch.zeros_like(p))
    if st["bias"] is None:
        key = l.double()
    else:                                      # values next to each other are told apart in 64 bits
        d = torch.where(on, l, torch.full_like(l, -1e30)).double()
        key = (torch.softmax(d, 1) if c["score"] == "softmax" else torch.sigmoid(d)) + st["bias"].double()
        key = torch.where(on, key, torch.full_like(key, float("-inf")))
    key, ids = torch.sort(key, dim=1, descending=True, stable=True)
    got = key[:, :k] > float("-inf")
    ids = ids[:, :k]
    s = torch.where(got, p.gather(1, ids), torch.zeros_like(p[:, :k]))
    total = s.sum(1, keepdim=True)
    w = s
    if c["normalize"]:
        w = torch.where(total > 0, s / total, torch.zeros_like(s))
    out = [torch.where(got, ids, torch.full_like(ids, -1)).to(torch.int32), w * c["scale"]]
    if c["grad"]:
        dw = torch.where(got, st["dweights"] * c["scale"], torch.zeros_like(s))
        if c["normalize"]:
            ds = dw - (w * dw).sum(1, keepdim=True)
            part = w * ds * (1 - s) if c["score"] == "sigmoid" else w * ds
            dl = torch.zeros_like(l).scatter_(1, ids, torch.where(got, part, torch.zeros_like(part)))
        elif c["score"] == "sigmoid":
            dl = torch.zeros_like(l).scatter_(1, ids, dw * s * (1 - s))
        else:
            dp = torch.zeros_like(l).scatter_(1, ids, dw)
            dl = p * (dp - (s * dw).sum(1, keepdim=True))
        out.append(dl.to(logits.dtype))
    return tuple(out)


def _plain_order(st):
    ids, first, G, rows = st["ids"], st["first"], st["G"], st["rows"]
    e = ids.reshape(-1).long() - first
    e = torch.where((e >= 0) & (e < G), e, torch.full_like(e, G))
    e, slot = torch.sort(e, stable=True)
    n = min(rows, e.numel())
    here = e[:n] < G
    slot_of = torch.full((rows,), -1, dtype=torch.int32, device=DEV)
    slot_of[:n] = torch.where(here, slot[:n], torch.full_like(slot[:n], -1)).to(torch.int32)
    row = torch.arange(e.numel(), device=DEV)
    row_of = torch.empty_like(row)
    row_of[slot] = torch.where((e < G) & (row < rows), row, torch.full_like(row, -1))
    ends = torch.searchsorted(e, torch.arange(G, device=DEV), right=True).clamp(max=rows)
    gs = torch.diff(ends, prepend=torch.zeros(1, dtype=ends.dtype, device=DEV))
    return gs.to(torch.int32), row_of.to(torch.int32).reshape(ids.shape), slot_of


def _taken(y, row_of):
    """Rows y[row_of] in fp32 [T,k,K], zeros where there is none."""
    r = row_of.long()
    v = y[r.clamp(min=0)].float()
    return torch.where((r >= 0)[:, :, None], v, torch.zeros_like(v))


def _placed(v, slot_of, k):
    """Rows [T,k,K] or tokens [T,K] in the sorted order, zeros where no slot owns the row."""
    s = slot_of.long()
    at = s.clamp(min=0)
    v = v.reshape(-1, v.shape[-1])[at] if v.dim() == 3 else v[at // k]
    return torch.where((s >= 0)[:, None], v, torch.zeros_like(v))


def _plain_move(st):
    gs, row_of, slot_of = _plain_order(st)
    x = _placed(st["x"], slot_of, st["case"]["k"])
    out = (st["weights"][:, :, None] * _taken(st["y"], row_of)).sum(1) + st["residual"].float()
    return gs, row_of, slot_of, x, out.to(st["y"].dtype)


def _plain_back(st):
    dt = st["y"].dtype
    dout, y = st["dout"].float(), _taken(st["y"], st["row_of"])
    dy = _placed((st["weights"][:, :, None] * dout[:, None, :]), st["slot_of"], st["case"]["k"])
    dweights = (dout[:, None, :] * y).sum(2)
    return dy.to(dt), dweights, _taken(st["drows"], st["row_of"]).sum(1).to(dt)


def _act(name, z):
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh((2 / math.pi) ** 0.5 * (z + 0.044715 * z ** 3)))
    return z


def _act_slope(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5
    if name == "gelu_tanh":
        c = (2 / math.pi) ** 0.5
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _groups(sizes):
    lo = 0
    for g, s in enumerate(sizes):
        if s:
            yield g, lo, lo + s
        lo += s


def _plain_linear(st):
    c, bf = st["case"], torch.bfloat16
    M, N = c["M"], c["N"]
    pre = torch.zeros((M, N), dtype=torch.float32, device=DEV)
    out = torch.zeros_like(pre)
    for g, lo, hi in _groups(st["sizes"]):
        z = st["x"][lo:hi].float() @ st["w"][g].float()
        if st["bias"] is not None:
            z = z + st["bias"][g].float()
        pre[lo:hi] = z
        out[lo:hi] = _act(c["act"], z)
        if st["residual"] is not None:
            out[lo:hi] += st["residual"][lo:hi].float()
    return (out.to(bf), pre.to(bf)) if c["pre"] else out.to(bf)


def _plain_linear_bwd(st):
    c, bf = st["case"], torch.bfloat16
    M, G, K, N = c["M"], c["G"], c["K"], c["N"]
    dx = torch.zeros((M, K), dtype=torch.float32, device=DEV)
    dw = torch.zeros((G, K, N), dtype=torch.float32, device=DEV)
    db = torch.zeros((G, N), dtype=torch.float32, device=DEV)
    for g, lo, hi in _groups(st["sizes"]):
        d = st["dout"][lo:hi].float()
        if st["pre"] is not None:
            d = d * _act_slope(c["act"], st["pre"][lo:hi].float())
        dx[lo:hi] = d @ st["w"][g].float().t()
        dw[g] = st["x"][lo:hi].float().t() @ d
        db[g] = d.sum(0)
    return dx.to(bf), dw.to(bf), db


# -------------------------------------------------- the framework's calls --

def _own(st):
    import moe_grouped_gemm_gmm_amd as gmm
    op, c = st["op"], st["case"]
    if op == "route":
        how = dict(score=c["score"], normalize=c["normalize"], scale=c["scale"])
        ids, weights = gmm.gmm_route(st["logits"], c["k"], bias=st["bias"], **how)
        if not c["grad"]:
            return ids, weights
        return ids, weights, gmm.gmm_route_bwd(st["dweights"], st["logits"], ids, **how)
    if op in ("plan", "move"):
        order = gmm.gmm_sort_tokens(st["ids"], st["G"], first=st["first"], rows=st["rows"])
        if op == "plan":
            return order
        gs, row_of, slot_of = order
        x = gmm.gmm_dispatch(st["x"], row_of, slot_of)
        out = gmm.gmm_combine(st["y"], row_of, weights=st["weights"], residual=st["residual"])
        return gs, row_of, slot_of, x, out
    if op == "back":
        dy, dweights = gmm.gmm_combine_bwd(st["dout"], st["y"], st["row_of"], st["slot_of"], st["weights"])
        return dy, dweights, gmm.gmm_combine(st["drows"], st["row_of"])
    if op == "linear":
        pre = torch.empty((c["M"], c["N"]), dtype=torch.bfloat16, device=DEV) if c["pre"] else None
        out = gmm.gmm_bf16_linear(st["x"], st["w"], st["gs"], bias=st["bias"], activation=c["act"],
                                  residual=st["residual"], pre=pre)
        return (out, pre) if c["pre"] else out
    return gmm.gmm_bf16_linear_bwd(st["dout"], st["w"], st["gs"], lhs=st["x"], pre=st["pre"], activation=c["act"])


def run(state):
    if own:
        return _own(state)
    op = state["op"]
    return dict(route=_plain_route, plan=_plain_order, move=_plain_move, back=_plain_back, linear=_plain_linear,
                linear_bwd=_plain_linear_bwd)[op](state)


# ------------------------------------------------------------------- work --

def work(case):
    op = case["op"]
    if op == "route":
        T, E, k, b = case["T"], case["E"], case["k"], 2 if case["dt"] == "bf16" else 4
        n = T * E * b + T * k * 8 + (E * 4 if case["bias"] else 0)
        if case["grad"]:                       # scores, ids and weight gradients in, score gradients out
            n += 2 * T * E * b + T * k * 8
        return dict(bytes=n, flops=T * E * (8 if case["grad"] else 4) + T * k * E)
    if op in ("plan", "move", "back"):
        T, k = case["T"], case["k"]
        _, G, rows = local(case)
        used = min(rows, (T - case["pad"]) * k // case["ranks"])
        order = 4 * (2 * T * k + rows + G)
        if op == "plan":
            return dict(bytes=order, flops=T * k)
        K, b = case["K"], 2 if case["dt"] == "bf16" else 4
        if op == "move":                       # x in, rows out; results, residual and weights in, tokens out
            return dict(bytes=order + K * b * (T + rows + used + 2 * T) + 4 * T * k, flops=2 * used * K)
        return dict(bytes=K * b * (T + used + rows + used + T) + 4 * (3 * T * k + rows), flops=4 * used * K)
    M, G, K, N = case["M"], case["G"], case["K"], case["N"]
    s = sizes(case)
    rows, busy = int(s.sum()), int((s > 0).sum())
    if op == "linear":
        n = rows * K * 2 + busy * K * N * 2 + M * N * 2
        n += (busy * N * 2 if case["bias"] else 0) + (rows * N * 2 if case["residual"] else 0)
        n += M * N * 2 if case["pre"] else 0
        return dict(bytes=n, flops=2 * rows * K * N)
    n = rows * N * 2 * (1 if case["act"] == "none" else 2) + rows * K * 2 + busy * K * N * 2
    return dict(bytes=n + M * K * 2 + G * K * N * 2 + G * N * 4, flops=4 * rows * K * N)


# ------------------------------------------------------ 64-bit definition --

def _exact_route(case, st):
    T, E, k, c = case["T"], case["E"], case["k"], case["scale"]
    l = st["logits"].to(torch.float64)
    off = l == float("-inf")
    if case["score"] == "softmax":
        top = l.max(dim=1, keepdim=True).values
        top = torch.where(top == float("-inf"), torch.zeros_like(top), top)
        s = torch.exp(l - top)
        s = s / s.sum(dim=1, keepdim=True).clamp(min=1e-300)
    else:
        s = 1 / (1 + torch.exp(-l))
    key = l.clone() if st["bias"] is None else (s + st["bias"].to(torch.float64)).masked_fill(off, float("-inf"))
    rows = torch.arange(T, device=DEV)
    ids = torch.full((T, k), -1, dtype=torch.int64, device=DEV)
    index = torch.arange(E, device=DEV).expand(T, E)
    for j in range(k):                         # the largest of what is left, the lowest of equals
        best = key.max(dim=1, keepdim=True).values
        at = torch.where(key == best, index, E).min(dim=1).values
        ok = best[:, 0] > float("-inf")
        ids[ok, j] = at[ok]
        key[rows[ok], at[ok]] = float("-inf")
    held = ids >= 0
    picked = torch.zeros((T, k), dtype=torch.float64, device=DEV)
    picked[held] = s[rows[:, None].expand(T, k)[held], ids[held]]
    total = picked.sum(dim=1, keepdim=True)
    w = c * picked / total.clamp(min=1e-300) if case["normalize"] else c * picked
    out = [ids.to(torch.int32), w]
    if case["grad"]:
        dw = torch.where(held, st["dweights"].to(torch.float64), 0.0)
        # of the scores, then through each score's own derivative
        ds = torch.zeros((T, E), dtype=torch.float64, device=DEV)
        if case["normalize"]:
            t = total.clamp(min=1e-300)
            g = c * (dw / t - (dw * picked).sum(dim=1, keepdim=True) / t ** 2)
        else:
            g = c * dw
        ds[rows[:, None].expand(T, k)[held], ids[held]] = g[held]
        if case["score"] == "softmax":
            out.append(s * (ds - (s * ds).sum(dim=1, keepdim=True)))
        else:
            out.append(ds * s * (1 - s))
    return tuple(out)


def _exact_order(case, ids):
    first, G, rows = local(case)
    flat = ids.cpu().numpy().reshape(-1)
    parts = [np.flatnonzero(flat == first + g) for g in range(G)]
    counts = np.array([p.size for p in parts])
    slots = np.concatenate(parts)[:rows]
    before = np.minimum(np.cumsum(counts) - counts, rows)
    gs = np.minimum(counts, rows - before)
    slot_of = np.full(rows, -1)
    slot_of[:slots.size] = slots
    row_of = np.full(flat.size, -1)
    row_of[slots] = np.arange(slots.size)
    t = lambda a: torch.from_numpy(a.astype(np.int32)).to(DEV)
    return t(gs), t(row_of).reshape(ids.shape), t(slot_of)


def _exact_rows(case, st):
    T, k = case["T"], case["k"]
    gs, row_of, slot_of = _exact_order(case, st["ids"])
    if st["op"] == "plan":
        return gs, row_of, slot_of
    D, K, rows = torch.float64, case["K"], slot_of.numel()
    used = slot_of[slot_of >= 0].long()
    n, token = used.numel(), used // k
    scale = st["weights"].to(D).reshape(-1)[used][:, None]
    if st["op"] == "move":
        x = torch.zeros((rows, K), dtype=D, device=DEV)
        x[:n] = st["x"].to(D)[token]
        out = st["residual"].to(D).clone()
        out.index_add_(0, token, scale * st["y"][:n].to(D))
        return gs, row_of, slot_of, x, out
    dy = torch.zeros((rows, K), dtype=D, device=DEV)
    d = st["dout"].to(D)[token]
    dy[:n] = scale * d
    dweights = torch.zeros(T * k, dtype=D, device=DEV)
    dweights[used] = (d * st["y"][:n].to(D)).sum(dim=1)
    dx = torch.zeros((T, K), dtype=D, device=DEV)
    dx.index_add_(0, token, st["drows"][:n].to(D))
    return dy, dweights.reshape(T, k), dx


def _exact_linear(case, st):
    D, M, G, K, N = torch.float64, case["M"], case["G"], case["K"], case["N"]
    edge = np.concatenate([[0], np.cumsum(st["sizes"])])
    a, root = case["act"], math.sqrt(2 / math.pi)

    def act_and_slope(z):
        if a == "none":
            return z, torch.ones_like(z)
        if a == "relu":
            return z.clamp(min=0), (z > 0).to(D)
        if a == "gelu":
            cdf = 0.5 * torch.special.erfc(-z / math.sqrt(2))
            return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        # silu, and the tanh form of gelu: z / (1 + exp(-u))
        u, du = (z, torch.ones_like(z)) if a == "silu" else \
            (2 * root * (z + 0.044715 * z ** 3), 2 * root * (1 + 0.134145 * z ** 2))
        s = 1 / (1 + torch.exp(-u))
        return z * s, s + z * s * (1 - s) * du

    if st["op"] == "linear":
        pre = torch.zeros((M, N), dtype=D, device=DEV)
        out = torch.zeros((M, N), dtype=D, device=DEV)
        for g in range(G):
            r = slice(int(edge[g]), int(edge[g + 1]))
            pre[r] = st["x"][r].to(D) @ st["w"][g].to(D) + (0 if st["bias"] is None else st["bias"][g].to(D))
            out[r] = act_and_slope(pre[r])[0] + (0 if st["residual"] is None else st["residual"][r].to(D))
        return (out, pre) if case["pre"] else out
    dx = torch.zeros((M, K), dtype=D, device=DEV)
    dw = torch.zeros((G, K, N), dtype=D, device=DEV)
    db = torch.zeros((G, N), dtype=D, device=DEV)
    for g in range(G):
        r = slice(int(edge[g]), int(edge[g + 1]))
        d = st["dout"][r].to(D)
        if st["pre"] is not None:
            d = d * act_and_slope(st["pre"][r].to(D))[1]
        dx[r] = d @ st["w"][g].to(D).T
        dw[g] = st["x"][r].to(D).T @ d
        db[g] = d.sum(dim=0)
    return dx, dw, db


def exact(case, seed):
    st = prepare(case, seed)
    if st["op"] == "route":
        return _exact_route(case, st)
    if st["op"] in ("plan", "move", "back"):
        return _exact_rows(case, st)
    return _exact_linear(case, st)
