"""GPU: the gated expert block and 8-bit checkpoints against plain 64-bit
computations written here.

Tolerances.  bf16 rounds by at most 2^-8 of the value, E4M3 by 2^-4 (half a
step of its subnormals, 2^-10 of the block scale, below 2^-6 of it).  A dot
product of n terms accumulated in fp32 is off by at most n 2^-23 times the sum
of its terms' magnitudes (each addition rounds or truncates within one fp32
step of the partial sum).  dP is rounded once to bf16 before the two products
of the backward pass, so these carry 2^-8 of the sum of their terms'
magnitudes besides their own rounding; two independent roundings spread evenly
over half a step make sqrt(2/3) 2^-8 of the norm, so the norm of the error
stays under 2^-8 of the gradient's."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_gmm_amd as gmm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
U = {BF: 2.0 ** -8, F32: 2.0 ** -24}

# sizes, M, K, N
SHAPES = [
    ([1], 1, 64, 64),                                     # one token, one expert
    ([0, 1, 0, 0], 1, 128, 64),
    ([3, 0, 1, 0, 2, 0, 0, 1], 8, 320, 192),              # a few rows, empty experts, unused row
    ([16, 17, 15, 1], 49, 192, 128),                      # around one 16-row tile
    ([33, 31, 0, 64, 65], 200, 128, 320),                 # around 32 and 64; unused rows
    ([127, 128, 129, 0, 1], 400, 256, 64),                # around one 128-row tile
    ([300, 0, 257, 255], 900, 448, 704),                  # several tiles, odd widths
    ([0, 0, 0], 70, 64, 128),                             # no rows at all
    ([700], 700, 1088, 192),
    ([2, 0, 5] * 50, 400, 64, 64),                        # more than 64 and 128 groups
    ([1, 0, 0, 2] * 100, 310, 128, 64),                   # more than 256 groups
]
IDS = ["M%d_K%d_N%d_G%d" % (M, K, N, len(s)) for s, M, K, N in SHAPES]


def normal(seed, shape, scale=1.0):
    r = np.random.default_rng([seed, 77])
    return torch.from_numpy((r.standard_normal(shape) * scale).astype(np.float32)).to(BF)


class Problem:
    def __init__(self, s, M, K, N, seed=0):
        self.s, self.M, self.K, self.N, self.G = s, M, K, N, len(s)
        self.used = sum(s)
        self.x = normal(seed, (M, K))
        self.w = normal(seed + 1, (self.G, K, 2 * N), K ** -0.5)
        self.dh = normal(seed + 2, (M, N), 0.5)
        self.gu = normal(seed + 3, (M, 2 * N), 1.5)
        for t in (self.x, self.dh, self.gu):
            t[self.used:] = float("nan")
        self.gs = torch.tensor(s, dtype=torch.int32, device=DEV)
        self.ends = np.concatenate([[0], np.cumsum(s)]).astype(int)

    def groups(self):
        for g in range(self.G):
            yield g, slice(self.ends[g], self.ends[g + 1])

    def dev(self, *names):
        return [getattr(self, n).to(DEV) for n in names]


def f64(t):
    return t.detach().cpu().double().numpy()


def silu(z):
    return z / (1 + np.exp(-z))


def forward64(p):
    """P and the sums of its terms' magnitudes, [M,2N] float64, zeros past the groups."""
    P, A = np.zeros((p.M, 2 * p.N)), np.zeros((p.M, 2 * p.N))
    x, w = f64(p.x), f64(p.w)
    for g, r in p.groups():
        P[r] = x[r] @ w[g]
        A[r] = np.abs(x[r]) @ np.abs(w[g])
    return P, A


def check(got, want, tol, name):
    got = f64(got)
    assert np.isfinite(got).all(), name
    bad = np.abs(got - want) > tol
    assert not bad.any(), "%s: %d of %d off, worst %g over its bound" % (
        name, bad.sum(), bad.size, (np.abs(got - want) - tol).max())


def h_bound(P, dP, N, u):
    g, up = P[:, :N], P[:, N:]
    h = silu(g) * up
    # |silu'| <= 1.1; exp, the division and the products: a few fp32 roundings of h
    return h, 1.1 * np.abs(up) * dP[:, :N] + 1.1 * np.abs(silu(g)) * dP[:, N:] + dP[:, :N] * dP[:, N:] \
        + (u + 2.0 ** -20) * np.abs(h) + 1e-37


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
@pytest.mark.parametrize("save", ["none", "bf16", "mx8"])
@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
def test_forward(shape, save, dt):
    p = Problem(*shape)
    x, w = p.dev("x", "w")
    M, N = p.M, p.N
    gu = torch.full((M, 2 * N), float("nan"), dtype=BF, device=DEV) if save == "bf16" else None
    q = torch.full((M, 2 * N), 0x55, dtype=torch.uint8, device=DEV) if save == "mx8" else None
    s = torch.full((M, 2 * N // 32), 0x55, dtype=torch.uint8, device=DEV) if save == "mx8" else None
    out = torch.full((M, N), float("nan"), dtype=dt, device=DEV)
    ws = gmm.workspace(gmm.OP_BF16_SWIGLU, M, p.K, N, p.G, DEV)
    assert gmm.gmm_bf16_swiglu(x, w, p.gs, out=out, gu=gu, gu_q=q, gu_scale=s, ws=ws) is out
    assert gmm.device_status(ws) == 0
    P, A = forward64(p)
    dP = p.K * 2.0 ** -23 * A
    h, tol = h_bound(P, dP, N, U[dt])
    check(out, h, tol, "h")
    assert (out[p.used:] == 0).all()
    if save == "bf16":
        check(gu, P, dP + U[BF] * np.abs(P), "P")
        assert (gu[p.used:] == 0).all()
    if save == "mx8":
        assert (q[p.used:] == 0).all() and (s[p.used:] == 0).all()
        v = gmm.gmm_dequantize_mx8(q, s, out_dtype=F32)
        scale = 2.0 ** (s.cpu().double().numpy() - 127).repeat(32, axis=1)
        check(v, P, 2.0 ** -4 * np.abs(P) + 2.0 ** -10 * scale + 1.1 * dP, "checkpoint of P")
        # the scale is the smallest that holds the block
        amax = np.abs(P).reshape(M, -1, 32).max(2)
        slack = 1 + 2.0 ** -10
        sc = 2.0 ** (s.cpu().double().numpy() - 127)
        live = amax > 0
        assert (amax[live] <= 448 * sc[live] * slack).all() and (amax[live] * slack > 224 * sc[live]).all()


def grad64(p, P):
    """dP, dx and dw in 64 bits, with the term-magnitude sums of dx and dw."""
    g, u, dh = P[:p.used, :p.N], P[:p.used, p.N:], f64(p.dh)[:p.used]
    s = 1 / (1 + np.exp(-g))
    d = np.concatenate([dh * u * s * (1 + g * (1 - s)), dh * g * s], axis=1)
    return d


def backward_check(p, x, d, dx, dw, h, P, dxt, dwt):
    w = f64(p.w)
    K, NN = p.K, 2 * p.N
    rdx, adx = np.zeros((p.M, K)), np.zeros((p.M, K))
    rdw, adw = np.zeros((p.G, K, NN)), np.zeros((p.G, K, NN))
    rows = np.array(p.s, dtype=float)[:, None, None]
    # d's fp32 evaluation cancels inside 1 + g (1 - s): bounded by a few fp32 steps of its terms, far under 2^-8
    for g, r in p.groups():
        rdx[r], adx[r] = d[r] @ w[g].T, np.abs(d[r]) @ np.abs(w[g]).T
        rdw[g], adw[g] = x[r].T @ d[r], np.abs(x[r]).T @ np.abs(d[r])
    ud = U[BF] + 2.0 ** -18
    if dx is not None:
        check(dx, rdx, (ud + NN * 2.0 ** -23) * adx * 1.01 + U[dxt] * np.abs(rdx) + 1e-30, "dx")
        assert np.linalg.norm(f64(dx) - rdx) <= 2.0 ** -8 * np.linalg.norm(rdx) + 1e-30
        assert (dx[p.used:] == 0).all()
    if dw is not None:
        check(dw, rdw, (ud + rows * 2.0 ** -23) * adw * 1.01 + U[dwt] * np.abs(rdw) + 1e-30, "dw")
        assert np.linalg.norm(f64(dw) - rdw) <= 2.0 ** -8 * np.linalg.norm(rdw) + 1e-30
        for g in range(p.G):
            if p.s[g] == 0:
                assert (dw[g] == 0).all()
    if h is not None:
        want = np.zeros((p.M, p.N))
        want[:p.used] = silu(P[:p.used, :p.N]) * P[:p.used, p.N:]
        check(h, want, (U[BF] + 2.0 ** -20) * np.abs(want) + 1e-37, "h recomputed")


def mx8_64(v):
    """Values, codes' scales of the 8-bit checkpoint of v [M,K], float64."""
    M, K = v.shape
    b = v.reshape(M, K // 32, 32)
    a = np.abs(b).max(2)
    m, e = np.frexp(a / 448)
    c = np.where(a == 0, -127, np.maximum(np.where(m == 0.5, e - 1, e), -127))
    y = b / np.exp2(c.astype(float))[:, :, None]
    _, k = np.frexp(y)
    step = np.exp2(np.maximum(k - 4, -9).astype(float))
    val = np.rint(y / step) * step
    return val.reshape(M, K), c + 127, (val * np.exp2(c.astype(float))[:, :, None]).reshape(M, K)


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "mx8"])
@pytest.mark.parametrize("dxt,dwt", [(BF, BF), (F32, F32)], ids=["bf16", "f32"])
def test_backward(shape, mx, dxt, dwt):
    p = Problem(*shape, seed=5)
    dh, w = p.dev("dh", "w")
    kw, x, P = {}, f64(p.x)[:p.used], f64(p.gu)
    if mx:
        _, _, xv = mx8_64(x)
        _, _, pv = mx8_64(np.nan_to_num(P))
        kw["lhs_q"], kw["lhs_scale"] = gmm.gmm_quantize_mx8(p.x.to(DEV))
        kw["gu_q"], kw["gu_scale"] = gmm.gmm_quantize_mx8(torch.nan_to_num(p.gu).to(DEV))
        for k in ("lhs_q", "lhs_scale", "gu_q", "gu_scale"):
            kw[k][p.used:] = 0xFF                       # NaN codes and scales past the groups
        x, P = xv, pv
    else:
        kw["lhs"], kw["gu"] = p.dev("x", "gu")
    h = torch.full((p.M, p.N), float("nan"), dtype=BF, device=DEV)
    dx = torch.full((p.M, p.K), float("nan"), dtype=dxt, device=DEV)
    dw = torch.full((p.G, p.K, 2 * p.N), float("nan"), dtype=dwt, device=DEV)
    ws = gmm.workspace(gmm.OP_BF16_SWIGLU_BWD, p.M, p.K, p.N, p.G, DEV)
    ws.fill_(0xFF)
    r = gmm.gmm_bf16_swiglu_bwd(dh, w, p.gs, dx=dx, dw=dw, h=h, ws=ws, **kw)
    assert r[0] is dx and r[1] is dw
    assert gmm.device_status(ws) == 0
    backward_check(p, x, grad64(p, P), dx, dw, h, P, dxt, dwt)


def test_backward_parts():
    """Each gradient on its own equals the same gradient of the whole call."""
    p = Problem([40, 0, 90, 7], 150, 192, 128, seed=9)
    dh, w, x, gu = p.dev("dh", "w", "x", "gu")
    dx, dw = gmm.gmm_bf16_swiglu_bwd(dh, w, p.gs, lhs=x, gu=gu)
    dx1, none = gmm.gmm_bf16_swiglu_bwd(dh, w, p.gs, gu=gu, want_dw=False)
    assert none is None and torch.equal(dx, dx1)
    none, dw1 = gmm.gmm_bf16_swiglu_bwd(dh, w, p.gs, lhs=x, gu=gu, want_dx=False)
    assert none is None and torch.equal(dw, dw1)
    h = torch.empty((p.M, p.N), dtype=BF, device=DEV)
    assert gmm.gmm_bf16_swiglu_bwd(dh, w, p.gs, gu=gu, h=h, want_dx=False, want_dw=False) == (None, None)
    g, u = f64(gu)[:p.used, :p.N], f64(gu)[:p.used, p.N:]
    check(h[:p.used], silu(g) * u, (U[BF] + 2.0 ** -20) * np.abs(silu(g) * u) + 1e-37, "h")
    assert (h[p.used:] == 0).all()


def test_gradients_against_differences():
    """dx and dw along a direction against central differences of the 64-bit loss sum(dh * h)."""
    p = Problem([13, 0, 20, 4], 37, 128, 64, seed=21)
    x, w, dh = p.dev("x", "w", "dh")
    gu = torch.empty((p.M, 2 * p.N), dtype=BF, device=DEV)
    gmm.gmm_bf16_swiglu(x, w, p.gs, gu=gu)
    dx, dw = gmm.gmm_bf16_swiglu_bwd(dh, w, p.gs, lhs=x, gu=gu, dx_dtype=F32, dw_dtype=F32)
    x64, w64, dh64 = f64(p.x), f64(p.w), f64(p.dh)

    def loss(xx, ww):
        t = 0.0
        for g, r in p.groups():
            P = xx[r] @ ww[g]
            t += (dh64[r] * silu(P[:, :p.N]) * P[:, p.N:]).sum()
        return t

    r = np.random.default_rng(3)
    for vx, vw in ((r.standard_normal(x64.shape), 0 * w64), (0 * x64, r.standard_normal(w64.shape))):
        e = 1e-5
        num = (loss(x64 + e * vx, w64 + e * vw) - loss(x64 - e * vx, w64 - e * vw)) / (2 * e)
        ana = (f64(dx) * vx).sum() + (f64(dw) * vw).sum()
        # P and dP are rounded to bf16, each by 2^-8 at most, and the signs of vx, vw do not know
        # those roundings: the error is 2 x 2^-8 of the norm of the summed terms, times 4 for its spread
        norm = np.linalg.norm(f64(dx) * vx) + np.linalg.norm(f64(dw) * vw)
        assert abs(num - ana) <= 4 * 2 * 2.0 ** -8 * norm + 1e-6 * abs(num)


# ------------------------------------------------------------ checkpoints --

def raw(q):
    return q.cpu().numpy().astype(np.int64)


def code_values(q):
    e, f = (q >> 3) & 15, q & 7
    v = np.where(e == 0, f * 2.0 ** -9, (1 + f / 8) * np.exp2(e.astype(float) - 7))
    return np.where(q >= 128, -v, v)


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,K", [(1, 32), (3, 96), (77, 704), (513, 2048), (1000, 32)])
def test_quantize(M, K, dt):
    r = np.random.default_rng([M, K])
    v = r.standard_normal((M, K)) * np.exp2(r.integers(-110, 110, (M, K // 32)).astype(float)).repeat(32, axis=1)
    v *= np.exp2(-r.integers(0, 12, (M, K)).astype(float))
    v[M // 2] = 0
    t = torch.from_numpy(v.astype(np.float32)).to(dt)
    val, c, back = mx8_64(f64(t))
    q, s = gmm.gmm_quantize_mx8(t.to(DEV))
    assert np.array_equal(raw(s), c)
    assert np.array_equal(code_values(raw(q)), val)
    assert np.array_equal(np.signbit(code_values(raw(q))) & (val != 0), np.signbit(val) & (val != 0))
    for od in (BF, F32):
        assert np.array_equal(f64(gmm.gmm_dequantize_mx8(q, s, out_dtype=od)), back)


def test_quantize_borders():
    """Block maxima on, just under and just over 448 * 2^e, every rounding
    border of E4M3, the largest and smallest floats."""
    top = np.float32(448.0)
    rows = []
    for e in (-100, -3, 0, 5, 100):
        for m in (np.nextafter(top, np.float32(0)), top, np.nextafter(top, np.float32(1e9))):
            b = np.zeros(32, np.float32)
            b[7] = -m
            b[8:12] = [m / 2, m / 3, m / 1000, -m / 30000]
            rows.append(np.ldexp(b, e).astype(np.float32))
    codes = code_values(np.arange(0, 0x7F))
    mids = (codes[1:] + codes[:-1]) / 2
    for chunk in (mids, np.nextafter(mids.astype(np.float32), np.float32(0)),
                  np.nextafter(mids.astype(np.float32), np.float32(1e9))):
        for i in range(0, len(chunk), 31):
            b = np.full(32, 448.0, np.float32)
            b[1:1 + len(chunk[i:i + 31])] = chunk[i:i + 31]
            rows.append(b)
    big = np.zeros(32, np.float32)
    big[0] = np.finfo(np.float32).max
    tiny = np.zeros(32, np.float32)
    tiny[0], tiny[1] = np.float32(2.0 ** -126), np.float32(2.0 ** -149)
    rows += [big, -big, tiny, np.zeros(32, np.float32)]
    v = np.stack(rows)
    val, c, back = mx8_64(v.astype(np.float64))
    q, s = gmm.gmm_quantize_mx8(torch.from_numpy(v).to(DEV))
    assert np.array_equal(raw(s), c)
    assert np.array_equal(code_values(raw(q)), val)
    with np.errstate(over="ignore"):      # 2^128, the nearest code to the largest float, reads back as infinity
        want = back.astype(np.float32).astype(np.float64)
    assert np.array_equal(f64(gmm.gmm_dequantize_mx8(q, s, out_dtype=F32)), want)


def test_quantize_nan_and_infinity():
    """NaN and infinity read back as NaN; a NaN leaves its block's scale and
    other codes alone, an infinity takes the scale 2^120."""
    r = np.random.default_rng(8)
    v = r.standard_normal((5, 128)).astype(np.float32)
    v[:, 3], v[:, 40], v[:, 70], v[:, 127] = 0.0, 0.0, 0.0, 0.0
    bad = v.copy()
    bad[:, 3], bad[:, 40], bad[:, 70], bad[:, 127] = np.nan, -np.nan, np.inf, -np.inf
    for dt in (BF, F32):
        q0, s0 = gmm.gmm_quantize_mx8(torch.from_numpy(v).to(DEV, dt))
        q, s = gmm.gmm_quantize_mx8(torch.from_numpy(bad).to(DEV, dt))
        back = f64(gmm.gmm_dequantize_mx8(q, s, out_dtype=F32))
        assert np.array_equal(np.isnan(back), ~np.isfinite(bad))
        keep = np.isfinite(bad[0, :64])
        assert np.array_equal(raw(s)[:, :2], raw(s0)[:, :2]) and (raw(s)[:, 2:] == 247).all()
        assert np.array_equal(raw(q)[:, :64][:, keep], raw(q0)[:, :64][:, keep])
        assert (np.nan_to_num(back[:, 64:]) == 0).all()


@pytest.mark.parametrize("shape", [(8, 2, 512, 128), (300, 3, 512, 192), (8000, 8, 1088, 512)],
                         ids=["few", "tiles", "load_waves"])
def test_forward_checkpoint_beside_a_nan(shape):
    """A NaN column of the weights: P's column is NaN in the checkpoint, and the
    scales and codes beside it are those of the same weights with zeros there."""
    M, G, K, N = shape
    r = np.random.default_rng(9)
    x = torch.from_numpy(r.standard_normal((M, K))).to(DEV, BF)
    w = torch.from_numpy(r.standard_normal((G, K, 2 * N)) / 32).to(DEV, BF)
    gs = torch.tensor([M // G] * G, dtype=torch.int32, device=DEV)
    cols = [5, 64 + 33, N + 18]
    got = []
    for fill in (0.0, float("nan")):
        w[:, :, cols] = fill
        q = torch.empty(M, 2 * N, dtype=torch.uint8, device=DEV)
        s = torch.empty(M, 2 * N // 32, dtype=torch.uint8, device=DEV)
        gmm.gmm_bf16_swiglu(x, w, gs, gu_q=q, gu_scale=s)
        got.append((raw(q)[:M // G * G], raw(s)[:M // G * G]))
    (q0, s0), (q1, s1) = got
    assert np.array_equal(s0, s1)
    assert ((q1[:, cols] & 0x7F) == 0x7F).all()
    keep = np.setdiff1d(np.arange(2 * N), cols)
    assert np.array_equal(q0[:, keep], q1[:, keep])


def test_dequantize_every_code():
    """All 254 finite codes under every scale whose values are normal bf16 numbers."""
    codes = np.array([c for c in range(256) if c & 0x7F != 0x7F] + [0, 0], dtype=np.uint8)     # 256 = 8 blocks
    scales = np.arange(10, 246, dtype=np.uint8)
    q = torch.from_numpy(np.tile(codes, (len(scales), 1))).to(DEV)
    s = torch.from_numpy(np.tile(scales[:, None], (1, 8))).to(DEV)
    want = code_values(codes.astype(np.int64))[None, :] * np.exp2(scales.astype(float) - 127)[:, None]
    for od in (BF, F32):
        assert np.array_equal(f64(gmm.gmm_dequantize_mx8(q, s, out_dtype=od)), want)


@pytest.mark.parametrize("dwt", [BF, F32], ids=["bf16", "f32"])
def test_weight_gradient_reads_exact_values(dwt):
    """dy = identity rows: dw holds the checkpoint's values themselves."""
    r = np.random.default_rng(4)
    M = K = N = 192
    q = torch.from_numpy(r.integers(0, 256, (M, K)).astype(np.uint8))
    q[(q & 0x7F) == 0x7F] = 0
    s = torch.from_numpy(r.integers(20, 235, (M, K // 32)).astype(np.uint8))
    dy = torch.eye(M, N, dtype=BF)
    gs = torch.tensor([M], dtype=torch.int32, device=DEV)
    dw = gmm.tgmm_mx8(q.to(DEV), s.to(DEV), dy.to(DEV), gs, out_dtype=dwt)
    want = code_values(raw(q)) * np.exp2(s.numpy().astype(float) - 127).repeat(32, axis=1)
    assert np.array_equal(f64(dw[0]), want.T)


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
@pytest.mark.parametrize("dwt", [BF, F32], ids=["bf16", "f32"])
def test_weight_gradient(shape, dwt):
    p = Problem(*shape, seed=31)
    q, s = gmm.gmm_quantize_mx8(torch.nan_to_num(p.x).to(DEV))
    q[p.used:] = 0x7F
    s[p.used:] = 0xFF
    dw = torch.full((p.G, p.K, p.N), float("nan"), dtype=dwt, device=DEV)
    gmm.tgmm_mx8(q, s, p.dh.to(DEV), p.gs, out=dw)
    _, _, x = mx8_64(np.nan_to_num(f64(p.x)))
    dy = np.nan_to_num(f64(p.dh))
    want, mag = np.zeros(dw.shape), np.zeros(dw.shape)
    for g, r in p.groups():
        want[g], mag[g] = x[r].T @ dy[r], np.abs(x[r]).T @ np.abs(dy[r])
    n = np.array(p.s, dtype=float)[:, None, None]
    check(dw, want, n * 2.0 ** -23 * mag + U[dwt] * np.abs(want) + 1e-30, "dw")


# -------------------------------------------------- the calls' contract ----

@pytest.mark.parametrize("sizes,M", [([160, 160, 40], 256), ([-7, 100, 60], 256), ([0, 300, -2, 50], 256),
                                     ([2, 3, -1, 9], 8)])
def test_sizes_outside_the_contract(sizes, M):
    """Rows are clipped, the status says so, nothing outside the buffers is read or written."""
    K, N, G = 128, 192, len(sizes)
    s = np.array(sizes)
    o = np.concatenate([[0], np.cumsum(np.maximum(s, 0))])
    clip = [int(v) for v in np.minimum(o[1:], M) - np.minimum(o[:-1], M)]
    status = (gmm.DEV_SUM_GT_M if o[-1] > M else 0) | (gmm.DEV_NEGATIVE_SIZE if (s < 0).any() else 0)
    p = Problem(clip, M, K, N, seed=41)
    gs = torch.tensor(sizes, dtype=torch.int32, device=DEV)
    pad = 300

    def guarded(t, fill):
        big = torch.full((t.shape[0] + 2 * pad,) + tuple(t.shape[1:]), fill, dtype=t.dtype, device=DEV)
        big[pad:pad + t.shape[0]] = t.to(DEV)
        return big, big[pad:pad + t.shape[0]]

    nan = float("nan")
    _, x = guarded(p.x, nan)
    _, dh = guarded(p.dh, nan)
    w = p.w.to(DEV)
    hb, h = guarded(torch.zeros(M, N, dtype=BF), 7.0)
    pb, gu = guarded(torch.zeros(M, 2 * N, dtype=BF), 7.0)
    xb, dx = guarded(torch.zeros(M, K, dtype=BF), 7.0)
    ws = gmm.workspace(gmm.OP_BF16_SWIGLU_BWD, M, K, N, G, DEV)
    gmm.gmm_bf16_swiglu(x, w, gs, out=h, gu=gu, ws=ws)
    assert gmm.device_status(ws) == status
    _, dw = gmm.gmm_bf16_swiglu_bwd(dh, w, gs, lhs=x, gu=gu, dx=dx, ws=ws)
    assert gmm.device_status(ws) == status
    for big in (hb, pb, xb):
        assert (big[:pad] == 7.0).all() and (big[pad + M:] == 7.0).all()
    P, A = forward64(p)
    dP = K * 2.0 ** -23 * A
    check(gu, P, dP + U[BF] * np.abs(P), "P")
    Pk = f64(gu)
    backward_check(p, f64(p.x)[:p.used], grad64(p, Pk), dx, dw, None, Pk, BF, BF)


def test_no_rows():
    w = normal(1, (3, 64, 128)).to(DEV)
    gs = torch.zeros(3, dtype=torch.int32, device=DEV)
    e = lambda c, t=BF: torch.empty((0, c), dtype=t, device=DEV)
    assert gmm.gmm_bf16_swiglu(e(64), w, gs).shape == (0, 64)
    dx, dw = gmm.gmm_bf16_swiglu_bwd(e(64), w, gs, lhs=e(64), gu=e(128))
    assert dx.shape == (0, 64) and (dw == 0).all()
    q, s = gmm.gmm_quantize_mx8(e(64))
    assert gmm.gmm_dequantize_mx8(q, s).shape == (0, 64)
    assert (gmm.tgmm_mx8(q, s, e(64), gs) == 0).all()


def test_extreme_gates():
    """exp overflows and underflows inside the activation: h and the gradients stay right and finite."""
    K = N = 64
    g = np.array([-300.0, -100.0, -89.0, -20.0, -1e-30, 0.0, 1e-30, 20.0, 89.0, 300.0, 1e4, -1e4])
    M = len(g)
    x = torch.zeros(M, K, dtype=BF)
    x[:, 0] = torch.from_numpy(g).to(BF)
    x[:, 1] = 1
    w = torch.zeros(1, K, 2 * N, dtype=BF)
    w[0, 0, :N] = 1
    w[0, 1, N:] = 2
    gs = torch.tensor([M], dtype=torch.int32, device=DEV)
    gu = torch.empty((M, 2 * N), dtype=BF, device=DEV)
    h = gmm.gmm_bf16_swiglu(x.to(DEV), w.to(DEV), gs, out_dtype=F32, gu=gu)
    z = f64(x[:, :1])
    with np.errstate(over="ignore"):
        want = np.broadcast_to(z / (1 + np.exp(-z)) * 2, (M, N))
        s = 1 / (1 + np.exp(-z))
    # where exp(-g) overflows h is 0: |g| |u| / 3.4e38 off at most
    check(h, want, 2.0 ** -20 * np.abs(want) + 2e-36, "h")
    dh = torch.ones((M, N), dtype=BF, device=DEV)
    dx, _ = gmm.gmm_bf16_swiglu_bwd(dh, w.to(DEV), gs, lhs=x.to(DEV), gu=gu, dx_dtype=F32)
    dg, du = 2 * s * (1 + z * (1 - s)), z * s
    want = np.zeros((M, K))
    want[:, :1], want[:, 1:2] = N * dg, 2 * N * du
    check(dx, want, 2.0 ** -7 * np.abs(want) + 1e-34, "dx")


def test_other_stream_and_repeat():
    """On another stream than the default one, and bit-identical across calls."""
    p = Problem([100, 0, 333, 67], 520, 256, 192, seed=51)
    x, w, dh = p.dev("x", "w", "dh")

    def run():
        q, s = gmm.gmm_quantize_mx8(x)
        gq = torch.empty((p.M, 2 * p.N), dtype=torch.uint8, device=DEV)
        gsc = torch.empty((p.M, 2 * p.N // 32), dtype=torch.uint8, device=DEV)
        h = gmm.gmm_bf16_swiglu(x, w, p.gs, gu_q=gq, gu_scale=gsc)
        h2 = torch.empty_like(h)
        dx, dw = gmm.gmm_bf16_swiglu_bwd(dh, w, p.gs, lhs_q=q, lhs_scale=s, gu_q=gq, gu_scale=gsc, h=h2)
        return [h, gq, gsc, dx, dw, h2, gmm.gmm_dequantize_mx8(q, s)[:p.used],
                gmm.tgmm_mx8(q, s, dh, p.gs)]

    a = run()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        b = run()
    st.synchronize()
    for u, v in zip(a, b):
        assert torch.equal(u, v)


def test_graph_replays():
    """One training step captured and replayed, with eager work in between, against the eager step."""
    p = Problem([100, 0, 333, 67], 520, 256, 192, seed=61)
    x, w, dh = p.dev("x", "w", "dh")
    M, N, K, G = p.M, p.N, p.K, p.G
    o = dict(h=torch.zeros((M, N), dtype=BF, device=DEV), gq=torch.zeros((M, 2 * N), dtype=torch.uint8, device=DEV),
             gsc=torch.zeros((M, N // 16), dtype=torch.uint8, device=DEV),
             dx=torch.zeros((M, K), dtype=BF, device=DEV), dw=torch.zeros((G, K, 2 * N), dtype=F32, device=DEV),
             h2=torch.zeros((M, N), dtype=BF, device=DEV), few=torch.zeros((4, N), dtype=BF, device=DEV))
    few_gs = torch.tensor([1, 0, 2, 1], dtype=torch.int32, device=DEV)

    def run():
        q, s = gmm.gmm_quantize_mx8(x)
        gmm.gmm_bf16_swiglu(x, w, p.gs, out=o["h"], gu_q=o["gq"], gu_scale=o["gsc"])
        gmm.gmm_bf16_swiglu_bwd(dh, w, p.gs, lhs_q=q, lhs_scale=s, gu_q=o["gq"], gu_scale=o["gsc"], dx=o["dx"],
                                dw=o["dw"], h=o["h2"])
        gmm.gmm_bf16_swiglu(x[:4], w, few_gs, out=o["few"])

    run()
    torch.cuda.synchronize()
    eager = {k: v.clone() for k, v in o.items()}
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        run()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            run()
    torch.cuda.synchronize()
    for rep in range(3):
        for v in o.values():
            v.zero_()
        run() if rep == 1 else None
        junk = (torch.randn(1 << 20, device=DEV) * 3).sum()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.isfinite(junk)
        for k, v in o.items():
            assert torch.equal(v, eager[k]), (rep, k)


@pytest.mark.slow
def test_offsets_past_32_bits():
    """Elements past 2^31 of the weights, of dw and of a checkpoint."""
    G, K, N = 530, 2048, 1024                               # G K 2N = 2.2e9
    sizes = [0] * G
    sizes[0], sizes[-1] = 3, 5
    p = Problem([3, 5], 8, K, N, seed=71)
    w = torch.zeros((G, K, 2 * N), dtype=BF, device=DEV)
    w[0], w[-1] = p.w[0].to(DEV), p.w[1].to(DEV)
    gs = torch.tensor(sizes, dtype=torch.int32, device=DEV)
    x, dh = p.dev("x", "dh")
    gu = torch.empty((8, 2 * N), dtype=BF, device=DEV)
    gmm.gmm_bf16_swiglu(x, w, gs, gu=gu)
    P, A = forward64(p)
    check(gu, P, K * 2.0 ** -23 * A + U[BF] * np.abs(P), "P")
    dx, dw = gmm.gmm_bf16_swiglu_bwd(dh, w, gs, lhs=x, gu=gu)
    Pk = f64(gu)
    assert (dw[1:-1] == 0).all()
    backward_check(p, f64(p.x), grad64(p, Pk), dx, torch.stack([dw[0], dw[-1]]), None, Pk, BF, BF)
    del w, dw
    M, K = 70000, 32768                                     # M K = 2.3e9
    big = torch.zeros((M, K), dtype=BF, device=DEV)
    big[-1] = normal(72, (K,)).to(DEV)
    q, s = gmm.gmm_quantize_mx8(big)
    back = gmm.gmm_dequantize_mx8(q, s)
    _, c, want = mx8_64(f64(big[-1:]))
    assert np.array_equal(f64(back[-1:]), want) and np.array_equal(raw(s[-1:]), c)
    assert (back[:-1] == 0).all()


# Few rows an expert: 16, 32 and 64-row tiles, 16 + 16 and 32 + 32 columns, K slices fewer than waves.
FEW = [
    ([1], 1, 64, 64), ([16], 16, 2048, 128), ([17, 0, 15], 40, 128, 64), ([40, 0], 40, 192, 320),
    ([64], 64, 448, 64), ([70, 3, 0, 100], 200, 320, 192), ([0, 9, 31, 0, 33], 100, 576, 256),
    ([5, 0, 1, 2] * 3, 30, 64, 1024),
]


@pytest.mark.parametrize("shape", FEW, ids=["M%d_K%d_N%d_G%d" % (M, K, N, len(s)) for s, M, K, N in FEW])
@pytest.mark.parametrize("save", ["none", "bf16", "mx8"])
@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
def test_forward_few_rows(shape, save, dt):
    test_forward(shape, save, dt)


# Grids large enough for the tiles of 256 columns (forward and dw; dX), full and partly filled.
WIDE = [
    ([2, 0, 5] * 50, 400, 64, 512),
    ([140, 3, 0, 200, 129] * 8, 3800, 128, 1344),
    ([140, 3, 0, 200, 129] * 8, 3800, 1344, 64),
]
WIDE_IDS = ["M%d_K%d_N%d_G%d" % (M, K, N, len(s)) for s, M, K, N in WIDE]


@pytest.mark.parametrize("shape", WIDE, ids=WIDE_IDS)
@pytest.mark.parametrize("save", ["none", "bf16", "mx8"])
@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
def test_forward_wide(shape, save, dt):
    test_forward(shape, save, dt)


@pytest.mark.parametrize("shape", WIDE, ids=WIDE_IDS)
@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "mx8"])
@pytest.mark.parametrize("dxt,dwt", [(BF, BF), (F32, F32)], ids=["bf16", "f32"])
def test_backward_wide(shape, mx, dxt, dwt):
    test_backward(shape, mx, dxt, dwt)


@pytest.mark.parametrize("shape", [([70, 0, 33] * 20, 2100, 256, 1088)], ids=["G60"])
@pytest.mark.parametrize("dwt", [BF, F32], ids=["bf16", "f32"])
def test_weight_gradient_wide(shape, dwt):
    test_weight_gradient(shape, dwt)


# Long reductions: the first forward and the first and last dX take the tiles with load waves, the others those of 128
# rows (every form of the load waves: test_gpu_ffn_forms.py).
LOADWAVES = [
    ([130, 100, 129, 0, 160, 161, 90, 31] * 3, 2500, 1088, 1088),      # forward: 24 groups, partial column tiles
    ([150, 65, 0, 33, 100], 360, 8256, 512),                           # many column tiles of dX, a partial one
    ([100] * 25, 2500, 1280, 1344),
]
LW_IDS = ["M%d_K%d_N%d_G%d" % (M, K, N, len(s)) for s, M, K, N in LOADWAVES]


@pytest.mark.parametrize("shape", LOADWAVES, ids=LW_IDS)
@pytest.mark.parametrize("save", ["none", "bf16", "mx8"])
@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
def test_forward_load_waves(shape, save, dt):
    test_forward(shape, save, dt)


@pytest.mark.parametrize("shape", LOADWAVES, ids=LW_IDS)
@pytest.mark.parametrize("dxt,dwt", [(BF, BF), (F32, F32)], ids=["bf16", "f32"])
def test_backward_load_waves(shape, dxt, dwt):
    test_backward(shape, False, dxt, dwt)


def test_expert_layer_example():
    """The example's training step: the gradients of both forms against a 64-bit layer.  Each value of a
    checkpoint is off by at most 2^-4, evenly spread over half a step (2^-4 / sqrt 3 of the norm, 0.036); P's
    enters dP twice over (gate and up), x's and h's the weight gradients: under 0.1 of the norm with room, and
    under 0.02 for the bfloat16 form, whose roundings are 2^-8."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_layer.py")
    spec = importlib.util.spec_from_file_location("expert_layer", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    rows, E, k, n, seed = 500, 6, 256, 128, 3
    plain, small = mod.run(rows, E, k, n, seed)
    assert plain["kept"] == rows * (k + 3 * n) * 2
    assert small["kept"] == rows * (k + 2 * n) * 33 // 32
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    r = lambda shape, s: torch.randn(shape, generator=gen, device=DEV, dtype=BF).mul_(s)
    sizes = torch.bincount(torch.randint(0, E, (rows,), generator=gen, device=DEV), minlength=E).cpu().tolist()
    x, dy = f64(r((rows, k), 1.0)), f64(r((rows, k), 0.1))
    wgu, wd = f64(r((E, k, 2 * n), k ** -0.5)), f64(r((E, n, k), n ** -0.5))
    dx, dwgu, dwd, lo = np.zeros((rows, k)), np.zeros((E, k, 2 * n)), np.zeros((E, n, k)), 0
    for e, s in enumerate(sizes):
        q = slice(lo, lo + s)
        lo += s
        P = x[q] @ wgu[e]
        g, u = P[:, :n], P[:, n:]
        sg = 1 / (1 + np.exp(-g))
        dh = dy[q] @ wd[e].T
        d = np.concatenate([dh * u * sg * (1 + g * (1 - sg)), dh * g * sg], axis=1)
        dx[q], dwgu[e], dwd[e] = d @ wgu[e].T, x[q].T @ d, (g * sg * u).T @ dy[q]
    for o, lim in ((plain, 0.02), (small, 0.1)):
        for got, want in zip(o["grads"], (dx, dwgu, dwd)):
            assert np.linalg.norm(f64(got) - want) <= lim * np.linalg.norm(want)


def test_load_waves_many_rounds():
    """Several items a workgroup: dX of 90 groups over many column tiles, with unused rows and empty groups."""
    s = [37, 0, 161, 5, 160, 90, 0, 64, 33] * 10
    p = Problem(s, sum(s) + 700, 2304, 512, seed=81)      # 9 column tiles
    dh, w, gu = p.dev("dh", "w", "gu")
    dx, _ = gmm.gmm_bf16_swiglu_bwd(dh, w, p.gs, gu=gu, want_dw=False)
    P = f64(p.gu)
    backward_check(p, f64(p.x)[:p.used], grad64(p, P), dx, None, None, P, BF, BF)


def test_load_waves_many_groups():
    """The same with more groups than the registers of one scan hold."""
    s = [57, 0, 90, 5, 96, 110, 0, 74, 53] * 30
    p = Problem(s, sum(s) + 100, 576, 512, seed=91)
    dh, w, gu = p.dev("dh", "w", "gu")
    dx, _ = gmm.gmm_bf16_swiglu_bwd(dh, w, p.gs, gu=gu, want_dw=False, dx_dtype=F32)
    P = f64(p.gu)
    backward_check(p, f64(p.x)[:p.used], grad64(p, P), dx, None, None, P, F32, BF)


# Many weight-gradient tiles, one a workgroup.
WGRAD = [
    # every part of a 64-row slice, empty groups, a half row tile and a partial column tile
    ([0, 1, 15, 16, 17, 31, 32, 33, 47, 48, 49, 63, 64, 65, 127, 128, 129, 193, 0, 300] * 2, 2740, 576, 448),
    # one group with most of the rows
    ([10, 0, 70] * 6 + [2000] + [10, 0, 70] * 7, 3100, 512, 512),
    ([5, 0, 0, 0, 90] * 50, 4750, 192, 512),              # 250 groups, most of them empty
]
WG_IDS = ["M%d_K%d_N%d_G%d" % (M, K, N, len(s)) for s, M, K, N in WGRAD]


@pytest.mark.parametrize("shape", WGRAD, ids=WG_IDS)
@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "mx8"])
@pytest.mark.parametrize("dxt,dwt", [(BF, BF), (F32, F32)], ids=["bf16", "f32"])
def test_backward_many_tiles(shape, mx, dxt, dwt):
    test_backward(shape, mx, dxt, dwt)


@pytest.mark.parametrize("shape", [(s, M, K, 2 * N) for s, M, K, N in WGRAD], ids=WG_IDS)
@pytest.mark.parametrize("dwt", [BF, F32], ids=["bf16", "f32"])
def test_weight_gradient_many_tiles(shape, dwt):
    test_weight_gradient(shape, dwt)
