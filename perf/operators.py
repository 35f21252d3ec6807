"""The expert layer's training and serving operators, as a user's program calls them.

Two things that belong together in one mixture-of-experts layer:

* the gated feed-forward block over rows sorted by expert,
      P = x . w[g],  w [G, K, 2N] with the gate columns first,
      h = silu(P[:, :N]) * P[:, N:],
  forward (with or without keeping P for the backward pass) and backward
  (dx and dw from dh);
* activation checkpoints in 8 bits: blocks of 32 consecutive values of a row
  share one power-of-two scale 2^e, e the smallest integer with
  max|v| <= 448 * 2^e, and every value is kept as the nearest E4M3 number of
  v / 2^e.  A checkpoint is written from a tensor or by the forward kernel
  and read by the backward pass.

Kinds of cases (case["op"]):
  swiglu   the gated block's forward; case["save"]: "none" (serving) or "bf16"
           (P is returned too)
  bwd      its backward pass from P kept in bfloat16: dx and dw
  ckpt     a checkpoint of x written and read back
  wgrad    the weight gradient x^T dy of every expert with x from a checkpoint
  step     forward and backward of the gated block with both checkpoints (x
           and P) in 8 bits: h, dx, dw
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda:0"
BLOCK = 32           # values that share a checkpoint scale
E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one token of a 256-expert model, top-8: eight experts read for one row each
        dict(name="fwd_one_token", op="swiglu", save="none", M=8, G=256, K=2048, N=512, tail=0, route="one", rseed=3),
        # a small serving batch on one of eight expert-parallel ranks
        dict(name="fwd_decode_batch", op="swiglu", save="none", M=203, G=32, K=2048, N=512, tail=0, route="zipf",
             rseed=5),
        # the expert-parallel shard's training forward
        dict(name="fwd_train_shard", op="swiglu", save="bf16", M=8192, G=32, K=2048, N=512, tail=0, route="uniform",
             rseed=7),
        # odd widths, empty experts, unused rows at the end of the buffer
        dict(name="fwd_odd", op="swiglu", save="bf16", M=1777, G=13, K=1088, N=704, tail=41, route="holes", rseed=11),
        # a few rows of a small model's backward pass
        dict(name="bwd_small", op="bwd", M=301, G=5, K=512, N=192, tail=0, route="uniform", rseed=13),
        # the shard's training backward
        dict(name="bwd_train_shard", op="bwd", M=8192, G=32, K=2048, N=512, tail=0, route="uniform", rseed=17),
        # a checkpoint of a few rows, and of the whole production batch
        dict(name="ckpt_small", op="ckpt", M=77, K=704),
        dict(name="ckpt_production", op="ckpt", M=65536, K=2048),
        # the output projection's weight gradient from a checkpoint: an odd one and the shard's
        dict(name="wgrad_odd", op="wgrad", M=999, G=7, K=640, N=448, tail=30, route="holes", rseed=19),
        dict(name="wgrad_shard", op="wgrad", M=8192, G=32, K=512, N=2048, tail=0, route="uniform", rseed=23),
        # forward and backward with 8-bit checkpoints: the shard, and all 256 experts under skewed routing
        dict(name="step_shard", op="step", M=8192, G=32, K=2048, N=512, tail=0, route="uniform", rseed=29),
        dict(name="step_production", op="step", M=65536, G=256, K=2048, N=512, tail=0, route="zipf", rseed=31),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["swiglu", "swiglu", "bwd", "ckpt", "wgrad", "step"])
    if op == "ckpt":
        return dict(op=op, M=_log_int(rng, 1, 65536), K=64 * _log_int(rng, 2, 32))
    limit = 65536 * 2048 * 512
    while True:
        c = dict(op=op, M=_log_int(rng, 1, 65536), G=_log_int(rng, 1, 256), K=64 * _log_int(rng, 2, 64),
                 N=64 * _log_int(rng, 1, 32), route=rng.choice(["uniform", "zipf", "holes", "one"]),
                 rseed=rng.randrange(1 << 30))
        # the unused rows of a fixed-size buffer: none, or up to a quarter of it
        c["tail"] = rng.choice([0, rng.randrange(0, max(1, c["M"] // 4))])
        if op == "swiglu":
            c["save"] = rng.choice(["none", "bf16"])
        if c["M"] * c["K"] * c["N"] <= limit and c["G"] * c["K"] * c["N"] <= 256 * 2048 * 512:
            return c


def sizes(case):
    """Rows of each expert: a property of the case (its routing)."""
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


# ----------------------------------------------------------------- inputs --

def _normal(gen, shape, scale=1.0):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16).mul_(scale)


def _activations(gen, M, K):
    """Hidden states: unit normals with a few channels that run 8 times larger."""
    x = _normal(gen, (M, K))
    hot = torch.randint(0, K, (max(1, K // 256),), generator=gen, device=DEV)
    x[:, hot] *= 8.0
    return x


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed) * 7919 + 17)
    op, M, K = case["op"], case["M"], case["K"]
    st = dict(op=op, x=_activations(gen, M, K))
    if op == "ckpt":
        if M > 2:
            st["x"][M // 2] = 0.0              # a padding token
        return st
    N, G = case["N"], case["G"]
    s = sizes(case)
    st.update(sizes=[int(v) for v in s], N=N, save=case.get("save"),
              gs=torch.tensor(s, dtype=torch.int32, device=DEV))
    used = int(s.sum())
    st["x"][used:] = float("nan")              # rows of the buffer that no expert owns
    if op == "wgrad":
        st["dy"] = _normal(gen, (M, N), 0.25)
        st["dy"][used:] = float("nan")
        q, e = _quantise(st.pop("x")[:used].float())
        st["x_q"] = torch.full((M, K), 0x7F, dtype=torch.uint8, device=DEV)
        st["x_s"] = torch.full((M, K // BLOCK), 255, dtype=torch.uint8, device=DEV)
        st["x_q"][:used] = q.view(torch.uint8)
        st["x_s"][:used] = (e + 127).to(torch.uint8)
        return st
    st["w"] = _normal(gen, (G, K, 2 * N), K ** -0.5)
    if op in ("bwd", "step"):
        st["dh"] = _normal(gen, (M, N), 0.25)
        st["dh"][used:] = float("nan")
    if op == "bwd":
        st["gu"] = _normal(gen, (M, 2 * N), 1.4)
        st["gu"][used:] = float("nan")
    return st


# ------------------------------------------------------------ plain forms --

def _pow2(e):
    """2^e as fp32 for integers e in [-127, 127], exactly (from its bits)."""
    e = e.to(torch.int32)
    return torch.where(e > -127, (e + 127) << 23, torch.full_like(e, 1 << 22)).view(torch.float32)


def _quantise(v):
    """Codes (E4M3) and exponents of the 1x32 blocks of v, fp32 [M, K]."""
    M, K = v.shape
    b = v.reshape(M, K // BLOCK, BLOCK)
    a = b.abs().amax(dim=2)
    m, p = torch.frexp(a)                      # 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, p - 9, p - 8).clamp(min=-127)
    e = torch.where(a == 0, torch.full_like(e, -127), e)
    q = (b * _pow2(-e)[:, :, None]).to(torch.float8_e4m3fn)
    return q.reshape(M, K), e


def _values(q, e):
    M, K = q.shape
    return (q.float().reshape(M, K // BLOCK, BLOCK) * _pow2(e)[:, :, None]).reshape(M, K)


def _round_trip(v):
    return _values(*_quantise(v))


def _groups(sizes):
    lo = 0
    for g, s in enumerate(sizes):
        if s:
            yield g, lo, lo + s
        lo += s


def _plain_forward(st):
    M, N = st["x"].shape[0], st["N"]
    p = torch.zeros((M, 2 * N), dtype=torch.float32, device=DEV)
    for g, lo, hi in _groups(st["sizes"]):
        p[lo:hi] = st["x"][lo:hi].float() @ st["w"][g].float()
    return torch.sigmoid(p[:, :N]) * p[:, :N] * p[:, N:], p


def _plain_backward(st, x, p):
    """dx, dw (fp32) from the kept activations x and p = (gate, up), fp32."""
    M, K = st["dh"].shape[0], st["w"].shape[1]
    N, G = st["N"], len(st["sizes"])
    dx = torch.zeros((M, K), dtype=torch.float32, device=DEV)
    dw = torch.zeros((G, K, 2 * N), dtype=torch.float32, device=DEV)
    for g, lo, hi in _groups(st["sizes"]):
        gate, up, dh = p[lo:hi, :N], p[lo:hi, N:], st["dh"][lo:hi].float()
        s = torch.sigmoid(gate)
        dp = torch.cat([dh * up * (s * (1 + gate * (1 - s))), dh * (gate * s)], dim=1)
        dx[lo:hi] = dp @ st["w"][g].float().t()
        dw[g] = x[lo:hi].t() @ dp
    return dx, dw


def _plain(st):
    op, bf = st["op"], torch.bfloat16
    if op == "swiglu":
        h, p = _plain_forward(st)
        return (h.to(bf), p.to(bf)) if st["save"] == "bf16" else h.to(bf)
    if op == "bwd":
        dx, dw = _plain_backward(st, st["x"].float(), st["gu"].float())
        return dx.to(bf), dw.to(bf)
    if op == "ckpt":
        return _round_trip(st["x"].float()).to(bf)
    if op == "wgrad":
        x = _values(st["x_q"].view(torch.float8_e4m3fn), st["x_s"].int() - 127)
        dw = torch.zeros((len(st["sizes"]), x.shape[1], st["N"]), dtype=torch.float32, device=DEV)
        for g, lo, hi in _groups(st["sizes"]):
            dw[g] = x[lo:hi].t() @ st["dy"][lo:hi].float()
        return dw.to(bf)
    h, p = _plain_forward(st)
    dx, dw = _plain_backward(st, _round_trip(st["x"].float()), _round_trip(p))
    return h.to(bf), dx.to(bf), dw.to(bf)


# -------------------------------------------------- the framework's calls --

def _own(st):
    import moe_grouped_gemm_gmm_amd as gmm
    op = st["op"]
    if op == "swiglu":
        if st["save"] == "none":
            return gmm.gmm_bf16_swiglu(st["x"], st["w"], st["gs"])
        gu = torch.empty((st["x"].shape[0], 2 * st["N"]), dtype=torch.bfloat16, device=DEV)
        return gmm.gmm_bf16_swiglu(st["x"], st["w"], st["gs"], gu=gu), gu
    if op == "bwd":
        return gmm.gmm_bf16_swiglu_bwd(st["dh"], st["w"], st["gs"], lhs=st["x"], gu=st["gu"])
    if op == "ckpt":
        return gmm.gmm_dequantize_mx8(*gmm.gmm_quantize_mx8(st["x"]))
    if op == "wgrad":
        return gmm.tgmm_mx8(st["x_q"], st["x_s"], st["dy"], st["gs"])
    M, N = st["x"].shape[0], st["N"]
    x_q, x_s = gmm.gmm_quantize_mx8(st["x"])
    gu_q = torch.empty((M, 2 * N), dtype=torch.uint8, device=DEV)
    gu_s = torch.empty((M, 2 * N // BLOCK), dtype=torch.uint8, device=DEV)
    h = gmm.gmm_bf16_swiglu(st["x"], st["w"], st["gs"], gu_q=gu_q, gu_scale=gu_s)
    dx, dw = gmm.gmm_bf16_swiglu_bwd(st["dh"], st["w"], st["gs"], lhs_q=x_q, lhs_scale=x_s,
                                     gu_q=gu_q, gu_scale=gu_s)
    return h, dx, dw


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------- work --

def work(case):
    op, M, K = case["op"], case["M"], case["K"]
    if op == "ckpt":   # bf16 in, codes and scales written and read, bf16 out
        return dict(bytes=M * K * 4 + 2 * (M * K + M * K // BLOCK), flops=4 * M * K)
    N, G = case["N"], case["G"]
    s = sizes(case)
    rows, busy = int(s.sum()), int((s > 0).sum())
    mx8 = lambda cols: rows * cols + rows * cols // BLOCK
    wbytes = busy * K * 2 * N * 2
    gemm = 2 * rows * K * 2 * N
    if op == "swiglu":
        keep = M * 2 * N * 2 if case["save"] == "bf16" else 0
        return dict(bytes=rows * K * 2 + wbytes + M * N * 2 + keep, flops=gemm)
    if op == "wgrad":
        return dict(bytes=mx8(K) + rows * N * 2 + G * K * N * 2, flops=2 * rows * K * N)
    # backward: dh, kept activations and weights in; dx and dw out
    back = rows * N * 2 + wbytes + M * K * 2 + G * K * 2 * N * 2
    if op == "bwd":
        return dict(bytes=back + rows * (K + 2 * N) * 2, flops=2 * gemm)
    # x and the weights read by the forward, h written; checkpoints written and read once each
    fwd = rows * K * 2 + wbytes + M * N * 2
    return dict(bytes=fwd + back + 2 * (mx8(K) + mx8(2 * N)), flops=3 * gemm)


# ------------------------------------------------------ 64-bit definition --

def _exact_pow2(k):
    """2^k as float64 for integers k, exactly."""
    return ((k.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_mx8(v):
    """The value every element of v (float64) has in an 8-bit checkpoint."""
    shape = v.shape
    b = v.reshape(-1, BLOCK)
    a = b.abs().max(dim=1, keepdim=True).values
    m, p = torch.frexp(a / E4M3_MAX)           # a / 448 = m 2^p, m in [1/2, 1)
    scale = _exact_pow2(torch.where(m == 0.5, p - 1, p).clamp(min=-127))
    scale = torch.where(a == 0, torch.ones_like(a), scale)
    y = b / scale
    _, k = torch.frexp(y)                      # |y| in [2^(k-1), 2^k): steps of 2^(k-4), 2^-9 below 2^-6
    step = _exact_pow2((k - 4).clamp(min=-9))
    return (torch.round(y / step) * step * scale).reshape(shape)


def exact(case, seed):
    st = prepare(case, seed)
    op, D = st["op"], torch.float64
    if op == "ckpt":
        return _exact_mx8(st["x"].to(D))
    starts = np.concatenate([[0], np.cumsum(st["sizes"])])
    M, G, K, N = case["M"], case["G"], case["K"], case["N"]
    used = int(starts[-1])
    zeros = lambda *shape: torch.zeros(shape, dtype=D, device=DEV)
    if op == "wgrad":
        q = st["x_q"][:used].to(torch.int64)   # sign, 4-bit exponent (bias 7), 3-bit fraction
        ex, fr = (q >> 3) & 15, (q & 7).to(D)
        mag = torch.where(ex == 0, fr * 2.0 ** -9, (1 + fr / 8) * _exact_pow2(ex - 7))
        x = torch.where(q >= 128, -mag, mag).reshape(used, K // BLOCK, BLOCK)
        x = (x * _exact_pow2(st["x_s"][:used].to(torch.int64) - 127)[:, :, None]).reshape(used, K)
        dw = zeros(G, K, N)
        for g in range(G):
            rows = slice(int(starts[g]), int(starts[g + 1]))
            dw[g] = x[rows].T @ st["dy"][rows].to(D)
        return dw
    x = st["x"][:used].to(D)
    if op in ("swiglu", "step"):
        P = zeros(M, 2 * N)
        for g in range(G):
            rows = slice(int(starts[g]), int(starts[g + 1]))
            P[rows] = x[rows] @ st["w"][g].to(D)
        h = P[:, :N] / (1 + torch.exp(-P[:, :N])) * P[:, N:]
        if op == "swiglu":
            return (h, P) if st["save"] == "bf16" else h
        x, P = _exact_mx8(x), _exact_mx8(P)
    else:
        P = st["gu"][:used].to(D)
    g_, u_, dh = P[:used, :N], P[:used, N:], st["dh"][:used].to(D)
    t = torch.exp(-g_)
    d = torch.empty((used, 2 * N), dtype=D, device=DEV)
    d[:, :N] = dh * u_ * (1 + t + g_ * t) / (1 + t) ** 2
    d[:, N:] = dh * g_ / (1 + t)
    dx, dw = zeros(M, K), zeros(G, K, 2 * N)
    for g in range(G):
        rows = slice(int(starts[g]), int(starts[g + 1]))
        dx[rows] = d[rows] @ st["w"][g].to(D).T
        dw[g] = x[rows].T @ d[rows]
    return (dx, dw) if op == "bwd" else (h, dx, dw)
