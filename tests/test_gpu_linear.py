"""GPU: the grouped product with bias, activation and residual, and its
gradient, against numpy in 64 bits.

Bounds (u = 2^-24, half a step of fp32; h half a step of the type stored).
The sum of K products and a bias in fp32 is off by at most (K + 2) u of the sum
of their magnitudes, whatever the order; act' is at most 1.13, so act(pre) by
1.13 times that.  An activation by itself is off by r u of its value, r = 16 + 8
min(100, c): c is how far an error of its exponential's argument is enlarged
(the argument itself; z^2 for the error function).  Slopes are sums of terms of at most
1.3 together and are off by 1.3 (r + 16) u.  dpre is rounded to bf16 before the
products (2^-8 of it), unless there is no activation.  Values below the smallest
normal number may be 0 (2^-126), and so may a sigmoid below it, the reciprocal of
an exponential past 2^126: z times it is off by |z| 2^-126 more.
"""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_gmm_amd as gmm
import moe_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
U, TINY = 2.0 ** -24, 2.0 ** -126
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


def n64(t):
    return t.double().cpu().numpy()


def half(dt):
    return torch.finfo(dt).eps / 2


def rnd(shape, dt, seed, scale=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dt)


def spread(M, G, seed, empty=0.3, tail=0):
    """Rows of each group: some get none, `tail` rows belong to no group."""
    r = np.random.default_rng(seed)
    p = (r.random(G) > empty) * r.random(G)
    p[r.integers(G)] += 0.5
    return r.multinomial(M - tail, p / p.sum()).astype(np.int64)


def groups(sizes):
    lo = 0
    for g, s in enumerate(sizes):
        yield g, slice(lo, lo + int(s))
        lo += int(s)


def enlarged(act, z):
    if act == "gelu":
        c = z * z
    elif act == "silu":
        c = np.abs(z)
    elif act == "gelu_tanh":
        c = 1.6 * np.abs(z) * (1 + 0.0447 * z * z)
    else:
        c = np.zeros_like(z)
    return 16 + 8 * np.minimum(100, c)


def problem(M, G, K, N, sizes, seed):
    x, w = rnd((M, K), BF, seed), rnd((G, K, N), BF, seed + 1, K ** -0.5)
    x[int(np.sum(sizes)):] = float("nan")
    return x, w


def check_fwd(M, G, K, N, sizes, act, bias_dt=BF, residual=True, keep=True, out_dt=BF, seed=1, gs=None, clipped=None):
    """clipped: the sizes the call is to read where gs breaks the contract."""
    x, w = problem(M, G, K, N, sizes, seed)
    b = None if bias_dt is None else rnd((G, N), bias_dt, seed + 2, 0.5)
    used = int(np.sum(sizes))
    res = rnd((M, N), out_dt, seed + 3) if residual else None
    if residual:
        res[used:] = float("inf")
    pre = torch.full((M, N), 9.0, dtype=BF, device=DEV) if keep else None
    gst = torch.tensor(sizes if gs is None else gs, dtype=I32, device=DEV)
    out = gmm.gmm_bf16_linear(x.to(DEV), w.to(DEV), gst, bias=None if b is None else b.to(DEV), activation=act,
                              residual=None if res is None else res.to(DEV), out_dtype=out_dt, pre=pre)
    torch.cuda.synchronize()
    assert out.dtype == out_dt and out.shape == (M, N)
    on, pn = n64(out), None if pre is None else n64(pre)
    assert not on[used:].any() and (pn is None or not pn[used:].any())
    xn, wn = n64(x), n64(w)
    for g, r in groups(sizes):
        if r.start == r.stop:
            continue
        bg = 0.0 if b is None else n64(b[g])
        z = xn[r] @ wn[g] + bg
        ez = (K + 2) * U * (np.abs(xn[r]) @ np.abs(wn[g]) + np.abs(bg))
        if pn is not None:
            assert np.all(np.abs(pn[r] - z) <= ez + half(BF) * (np.abs(z) + ez) + TINY), "pre of group %d" % g
        v, _ = ref.act(act, z)
        rs = 0.0 if res is None else n64(res[r])
        e = 1.13 * ez + enlarged(act, z) * U * np.abs(v) + U * (np.abs(v) + np.abs(rs))
        assert np.all(np.abs(on[r] - (v + rs)) <= e + half(out_dt) * (np.abs(v + rs) + e) + TINY), "out of group %d" % g
    return out


# few rows (16, 32, 64; narrow and wide tiles), 128 and 256 columns, odd widths, many experts
SHAPES = [(1, 1, 64, 64), (8, 256, 512, 2048), (3, 300, 128, 64), (20, 2, 192, 128), (60, 3, 64, 320), (200, 5, 320, 192),
          (250, 40, 512, 1024), (1000, 30, 1088, 704), (777, 3, 704, 64), (2500, 9, 256, 1024), (600, 300, 64, 128),
          (4096, 4, 512, 2048)]


@pytest.mark.parametrize("M,G,K,N", SHAPES)
@pytest.mark.parametrize("act", ACTS)
def test_forward(M, G, K, N, act):
    i = ACTS.index(act)
    check_fwd(M, G, K, N, spread(M, G, M + i, tail=M // 10), act, bias_dt=[BF, F32, None][(M + i) % 3],
              residual=(M + i) % 2 == 0, keep=i != 1, out_dt=[BF, F32][(M // 2 + i) % 2], seed=10 * M + i)


@pytest.mark.parametrize("M,G,K,N", [(40, 3, 128, 192), (900, 4, 320, 448)])
def test_every_combination_of_operands(M, G, K, N):
    s = spread(M, G, 5, tail=7)
    for bias_dt in (None, BF, F32):
        for residual in (False, True):
            for keep in (False, True):
                for out_dt in (BF, F32):
                    check_fwd(M, G, K, N, s, "gelu", bias_dt, residual, keep, out_dt)


def test_no_rows_and_empty_groups():
    for M, sizes in ((0, [0, 0, 0]), (70, [0, 0, 0]), (70, [0, 70, 0]), (70, [1, 0, 1])):
        check_fwd(M, 3, 128, 128, sizes, "silu")


@pytest.mark.parametrize("M,K,N", [(60, 128, 128), (700, 128, 256)])
def test_sizes_outside_the_contract(M, K, N):
    """A negative size is read as 0, rows past M are clipped, and the status word tells."""
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    x, w = problem(M, 3, K, N, [M], 3)
    for gs, status, same in (([-4, 30, M], gmm.DEV_SUM_GT_M | gmm.DEV_NEGATIVE_SIZE, [0, 30, M - 30]),
                             ([M, 5, 2 ** 31 - 1], gmm.DEV_SUM_GT_M, [M, 0, 0]), ([10, -1, 20], gmm.DEV_NEGATIVE_SIZE, [10, 0, 20])):
        t = lambda v: torch.tensor(v, dtype=I32, device=DEV)
        a = gmm.gmm_bf16_linear(x.to(DEV), w.to(DEV), t(gs), activation="relu", ws=ws)
        assert gmm.device_status(ws) == status
        assert torch.equal(a, gmm.gmm_bf16_linear(x.to(DEV), w.to(DEV), t(same), activation="relu"))


def test_residual_in_place_and_outputs_given():
    M, G, K, N = 300, 4, 128, 192
    s = spread(M, G, 2, tail=20)
    x, w = problem(M, G, K, N, s, 4)
    gs = torch.tensor(s, dtype=I32, device=DEV)
    r = rnd((M, N), BF, 7).to(DEV)
    want = gmm.gmm_bf16_linear(x.to(DEV), w.to(DEV), gs, residual=r)
    assert gmm.gmm_bf16_linear(x.to(DEV), w.to(DEV), gs, residual=r, out=r) is r and torch.equal(r, want)
    big = torch.full((M + 4, N), 7.0, dtype=BF, device=DEV)
    gmm.gmm_bf16_linear(x.to(DEV), w.to(DEV), gs, out=big[2:M + 2])
    assert (big[:2] == 7).all() and (big[M + 2:] == 7).all()


def test_tails_of_the_activations():
    """Small results keep their digits: identity weights, one row of arguments from -20 to 20."""
    N = 512
    z = torch.linspace(-20, 20, N).to(BF)
    x, w = z.reshape(1, N).to(DEV), torch.eye(N, dtype=BF, device=DEV).reshape(1, N, N)
    gs = torch.ones(1, dtype=I32, device=DEV)
    zn = n64(z)
    for act in ACTS:
        got = n64(gmm.gmm_bf16_linear(x, w, gs, activation=act, out_dtype=F32))[0]
        v, _ = ref.act(act, zn)
        assert np.all(np.abs(got - v) <= enlarged(act, zn) * U * np.abs(v) + TINY * (1 + np.abs(zn))), act


def check_bwd(M, G, K, N, sizes, act, dx_dt=BF, dw_dt=BF, db_dt=F32, seed=1):
    used = int(np.sum(sizes))
    x, w = problem(M, G, K, N, sizes, seed)
    dout, pre = rnd((M, N), BF, seed + 2), rnd((M, N), BF, seed + 3, 1.5)
    dout[used:], pre[used:] = float("nan"), float("nan")
    gs = torch.tensor(sizes, dtype=I32, device=DEV)
    pd = None if act == "none" else pre.to(DEV)
    args = (dout.to(DEV), w.to(DEV), gs)
    dx, dw, db = gmm.gmm_bf16_linear_bwd(*args, lhs=x.to(DEV), pre=pd, activation=act, dx_dtype=dx_dt, dw_dtype=dw_dt,
                                         db_dtype=db_dt)
    torch.cuda.synchronize()
    assert (dx.dtype, dw.dtype, db.dtype) == (dx_dt, dw_dt, db_dt)
    xn, wn, dn, zn = n64(x), n64(w), n64(dout), n64(pre)
    dxn, dwn, dbn = n64(dx), n64(dw), n64(db)
    assert not dxn[used:].any()
    for g, r in groups(sizes):
        n = r.stop - r.start
        if n == 0:
            assert not dwn[g].any() and not dbn[g].any()
            continue
        d, e0, e1 = dn[r], np.zeros((n, N)), np.zeros((n, N))
        if act != "none":
            d = dn[r] * ref.act(act, zn[r])[1]
            e0 = 1.3 * (enlarged(act, zn[r]) + 16) * U * np.abs(dn[r]) + TINY   # of dpre in fp32
            e1 = e0 + half(BF) * (np.abs(d) + e0)                               # and rounded
        a = np.abs(d) + e1
        for got, want, e, dt in ((dxn[r], d @ wn[g].T, e1 @ np.abs(wn[g]).T + N * U * (a @ np.abs(wn[g]).T), dx_dt),
                                 (dwn[g], xn[r].T @ d, np.abs(xn[r]).T @ e1 + n * U * (np.abs(xn[r]).T @ a), dw_dt),
                                 (dbn[g], d.sum(0), e0.sum(0) + (n + 2) * U * a.sum(0), db_dt)):
            assert np.all(np.abs(got - want) <= e + half(dt) * (np.abs(want) + e) + TINY), "group %d" % g
    # each alone gives the same
    for k, want in enumerate((dx, dw, db)):
        got = gmm.gmm_bf16_linear_bwd(*args, lhs=x.to(DEV) if k == 1 else None, pre=pd, activation=act, dx_dtype=dx_dt,
                                      dw_dtype=dw_dt, db_dtype=db_dt, want_dx=k == 0, want_dw=k == 1, want_db=k == 2)
        assert [o is None for o in got] == [k != 0, k != 1, k != 2] and torch.equal(got[k], want)
    return dx, dw, db


@pytest.mark.parametrize("M,G,K,N", [(1, 1, 64, 64), (8, 256, 128, 512), (60, 3, 64, 320), (301, 5, 512, 192), (777, 3, 704, 64),
                                     (1000, 13, 1088, 704), (2500, 9, 256, 1024), (600, 300, 64, 128), (333, 2, 64, 4160)])
@pytest.mark.parametrize("act", ACTS)
def test_backward(M, G, K, N, act):
    i = ACTS.index(act)
    check_bwd(M, G, K, N, spread(M, G, M + i, tail=M // 10), act, [BF, F32][i % 2], [F32, BF][i % 2 if M % 2 else 0],
              [F32, BF][(M + i) % 2], seed=10 * M + i)


def test_backward_of_no_rows():
    for M, sizes in ((0, [0, 0, 0]), (70, [0, 0, 0]), (70, [0, 70, 0])):
        for act in ("none", "gelu"):
            check_bwd(M, 3, 128, 128, sizes, act)


def test_gradient_against_differences():
    """The backward pass is that of what the forward computes: directional differences of the forward in fp32."""
    M, G, K, N = 96, 3, 128, 128
    s = [40, 0, 56]
    gs = torch.tensor(s, dtype=I32, device=DEV)
    x, w = rnd((M, K), BF, 1).to(DEV), rnd((G, K, N), BF, 2, K ** -0.5).to(DEV)
    b, v = rnd((G, N), F32, 3, 0.5).to(DEV), rnd((M, N), BF, 4).to(DEV)
    dirb = rnd((G, N), F32, 5).to(DEV)
    for act in ("silu", "gelu", "gelu_tanh"):
        pre = torch.empty((M, N), dtype=BF, device=DEV)
        gmm.gmm_bf16_linear(x, w, gs, bias=b, activation=act, pre=pre)
        _, _, db = gmm.gmm_bf16_linear_bwd(v, w, gs, lhs=x, pre=pre, activation=act)
        h = 1.0 / 64
        f = lambda t: (gmm.gmm_bf16_linear(x, w, gs, bias=b + t * dirb, activation=act, out_dtype=F32).double()
                       * v.double()).sum()
        num, ana = ((f(h) - f(-h)) / (2 * h)).item(), (db.double() * dirb.double()).sum().item()
        # pre kept in bf16 moves each slope by up to 2^-8 |z| times a curvature below 1, at random; h^2 third derivatives
        size = (v.double().abs() * pre.double().abs()).norm().item() + v.double().norm().item()
        assert abs(num - ana) <= 4 * size * (2.0 ** -8 + h * h), (act, num, ana)


def test_calls_repeat_and_streams_do_not_meet():
    M, G, K, N = 2000, 16, 256, 512
    s = spread(M, G, 9)
    gs = torch.tensor(s, dtype=I32, device=DEV)
    x, w = problem(M, G, K, N, s, 5)
    x, w = x.to(DEV), w.to(DEV)
    d, pre = rnd((M, N), BF, 8).to(DEV), rnd((M, N), BF, 9).to(DEV)
    run = lambda: (gmm.gmm_bf16_linear(x, w, gs, activation="gelu", residual=d),) + gmm.gmm_bf16_linear_bwd(
        d, w, gs, lhs=x, pre=pre, activation="gelu")
    want = run()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for _ in range(2):
        for st in streams:
            with torch.cuda.stream(st):
                got.append(run())
    torch.cuda.synchronize()
    for o in got:
        assert all(torch.equal(a, b) for a, b in zip(o, want))
