"""GPU: the gated block's kernels for large grids (tiles fed by load waves) in
every item height and round count that their rule can choose, each problem with
the kernel it is meant for asked from gmm_get_tile_config first, against the
64-bit computations and tolerances of test_gpu_ffn.py.

dP, the operand of both products of the backward pass, is rounded to bf16.
Against gradients of a dP rounded in the 64-bit computation too, what remains
is the fp32 evaluation: it moves a value by at most 2^-18 of its terms, so at
most 2 x 2^-18 / 2^-8 = 2^-9 of the values round to the other neighbour, by at
most 2^-7; the norm of that is sqrt(2^-9) 2^-7, under 2^-11 of dP's, and twice
that bounds the products."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_gmm_amd as gmm
import test_gpu_ffn as T

pytestmark = pytest.mark.gpu
DEV = T.DEV
BF, F32, U8 = T.BF, T.F32, torch.uint8
LOAD_WAVES = 3

_R = np.random.default_rng(12)
# name: sizes, M, K, N, item rows of the forward and of dX (0: another kernel)
FORMS = {
    # items of 129 to 160 rows: five 32-row blocks, three of them one wave's; 161 and more: two items
    "tall": ([160, 129, 145, 0, 158, 131, 160, 161, 140, 150, 33, 130] * 2, 3050, 832, 1088, 160, 96),
    # the same grid when one group has most of the rows (many more items than the host expects)
    "skewed": ([2000] + [20, 0, 1, 33] * 5 + [64, 96, 160], 3050, 832, 1088, 160, 96),
    # no group has any row: the whole buffer is unused
    "unused": ([0] * 24, 3050, 832, 1088, 160, 96),
    # two rounds of the chip, two items a group
    "two_rounds": ([250, 128, 129, 256, 0, 300, 190, 200, 31, 255] * 4, 7000, 2048, 576, 128, 160),
    # more groups than one scan keeps in registers
    "many_groups": ([int(v) for v in _R.integers(0, 140, 390)], 39000, 2048, 128, 128, 0),
    # short items
    "flat": ([96, 97, 192, 150, 0, 193, 170, 64, 146, 180, 33, 288] * 2, 3500, 1088, 512, 96, 96),
    "odd": ([200, 0, 129, 128, 127, 64, 65, 0, 300, 191, 33, 96, 320], 1777, 1088, 704, 64, 64),
}


def problem(name, seed=0):
    sizes, M, K, N = FORMS[name][:4]
    return T.Problem(sizes, M, K, N, seed=seed)


def chosen(name):
    """Item rows of the forward's and dX's load-wave tiles, 0 where another kernel runs."""
    sizes, M, K, N = FORMS[name][:4]
    got = [gmm.get_tile_config(op, M, K, N, len(sizes)) for op in (gmm.OP_BF16_SWIGLU, gmm.OP_BF16_SWIGLU_BWD)]
    return tuple(c["tile_m"] if c["kernel"] == LOAD_WAVES else 0 for c in got)


# every kind of P with every output type; one of each for the large problem
FORWARD = [(n, save, dt) for n in FORMS for save in ("none", "bf16", "mx8") for dt in (BF, F32)
           if n != "many_groups" or (save == "bf16") == (dt == F32)]


@pytest.mark.parametrize("name,save,dt", FORWARD, ids=["%s-%s-%s" % (n, s, "bf16" if d == BF else "f32")
                                                       for n, s, d in FORWARD])
def test_forward(name, save, dt):
    assert chosen(name)[0] == FORMS[name][4]
    T.test_forward(FORMS[name][:4], save, dt)


# Few rows an expert on grids too large for 16 + 16 columns a tile: sizes, M, K, N, tile rows.
FEW = {
    "rows_16": ([3, 0, 16, 17, 1] * 6, 300, 320, 512, 16),
    "rows_32": ([17, 32, 0, 33, 5] * 4, 450, 320, 512, 32),
    "rows_64": ([64, 65, 0, 63, 5, 100] * 3, 1000, 192, 576, 64),
}


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("save", ["none", "bf16", "mx8"])
@pytest.mark.parametrize("name", list(FEW))
def test_forward_few_rows(name, save, dt):
    sizes, M, K, N, rows = FEW[name]
    c = gmm.get_tile_config(gmm.OP_BF16_SWIGLU, M, K, N, len(sizes))
    assert (c["kernel"], c["tile_m"], c["tile_n"]) == (1, rows, 64)
    T.test_forward(FEW[name][:4], save, dt)


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("name", [n for n in FORMS if FORMS[n][5]])
def test_dx(name, dt):
    assert chosen(name)[1] == FORMS[name][5]
    p = problem(name, seed=5)
    dh, w, gu = p.dev("dh", "w", "gu")
    dx = torch.full((p.M, p.K), float("nan"), dtype=dt, device=DEV)
    gmm.gmm_bf16_swiglu_bwd(dh, w, p.gs, gu=gu, dx=dx, want_dw=False)
    P = T.f64(p.gu)
    w64, d = T.f64(p.w), T.grad64(p, P)
    want, mag = np.zeros((p.M, p.K)), np.zeros((p.M, p.K))
    for g, r in p.groups():
        want[r], mag[r] = d[r] @ w64[g].T, np.abs(d[r]) @ np.abs(w64[g]).T
    ud = T.U[BF] + 2.0 ** -18
    T.check(dx, want, (ud + 2 * p.N * 2.0 ** -23) * mag * 1.01 + T.U[dt] * np.abs(want) + 1e-30, "dx")
    assert (dx[p.used:] == 0).all()


@pytest.mark.parametrize("sizes", [[160, 200, -3, 0, 150] * 4 + [7, 0, 3000, 50],       # past M, and negative
                                   [120, 0, -7, 161] * 6,                              # negative
                                   [400] * 24], ids=["both", "negative", "sum"])
def test_sizes_outside_the_contract(sizes):
    """Rows are clipped, the status says so, nothing outside the buffers is written."""
    M, K, N = FORMS["tall"][1:4]
    assert chosen("tall") == FORMS["tall"][4:] and len(sizes) == 24
    s = np.array(sizes)
    o = np.concatenate([[0], np.cumsum(np.maximum(s, 0))])
    clip = [int(v) for v in np.minimum(o[1:], M) - np.minimum(o[:-1], M)]
    status = (gmm.DEV_SUM_GT_M if o[-1] > M else 0) | (gmm.DEV_NEGATIVE_SIZE if (s < 0).any() else 0)
    p = T.Problem(clip, M, K, N, seed=41)
    gs = torch.tensor(sizes, dtype=torch.int32, device=DEV)
    pad = 200

    def guarded(cols, dt, fill):
        big = torch.full((M + 2 * pad, cols), fill, dtype=dt, device=DEV)
        return big, big[pad:pad + M]

    # inputs surrounded by NaN: a row read past the clipped ones would show
    xb, x = guarded(K, BF, float("nan"))
    db, dh = guarded(N, BF, float("nan"))
    x.copy_(p.x)
    dh.copy_(p.dh)
    w = p.w.to(DEV)
    hb, h = guarded(N, BF, 7.0)
    gb, gu = guarded(2 * N, BF, 7.0)
    qb, q = guarded(2 * N, U8, 9)
    sb, sc = guarded(2 * N // 32, U8, 9)
    dxb, dx = guarded(K, BF, 7.0)
    ws = gmm.workspace(gmm.OP_BF16_SWIGLU_BWD, M, K, N, 24, DEV)
    gmm.gmm_bf16_swiglu(x, w, gs, out=h, gu_q=q, gu_scale=sc, ws=ws)
    assert gmm.device_status(ws) == status
    h2 = h.clone()
    gmm.gmm_bf16_swiglu(x, w, gs, out=h, gu=gu, ws=ws)
    assert gmm.device_status(ws) == status and torch.equal(h, h2)
    gmm.gmm_bf16_swiglu_bwd(dh, w, gs, gu=gu, dx=dx, want_dw=False, ws=ws)
    assert gmm.device_status(ws) == status
    for big, v in ((hb, 7.0), (gb, 7.0), (dxb, 7.0), (qb, 9), (sb, 9)):
        assert (big[:pad] == v).all() and (big[pad + M:] == v).all()
    P, A = T.forward64(p)
    dP = K * 2.0 ** -23 * A
    T.check(gu, P, dP + T.U[BF] * np.abs(P), "P")
    want, tol = T.h_bound(P, dP, N, T.U[BF])
    T.check(h, want, tol, "h")
    assert (h[p.used:] == 0).all() and (q[p.used:] == 0).all() and (sc[p.used:] == 0).all()
    Pk = T.f64(gu)
    T.backward_check(p, T.f64(p.x)[:p.used], T.grad64(p, Pk), dx, None, None, Pk, BF, BF)


def _step(p, x, w, dh, o):
    """Forward with each kind of P, and dX, into the tensors of o."""
    gmm.gmm_bf16_swiglu(x, w, p.gs, out=o["h"], gu=o["gu"])
    gmm.gmm_bf16_swiglu(x, w, p.gs, out=o["h32"], gu_q=o["q"], gu_scale=o["s"])
    gmm.gmm_bf16_swiglu(x, w, p.gs, out=o["h0"])
    gmm.gmm_bf16_swiglu_bwd(dh, w, p.gs, gu=o["gu"], dx=o["dx"], want_dw=False)
    gmm.gmm_bf16_swiglu_bwd(dh, w, p.gs, gu_q=o["q"], gu_scale=o["s"], dx=o["dx32"], want_dw=False)


def _outputs(p):
    e = lambda c, t: torch.full((p.M, c), 3, dtype=t, device=DEV)
    return dict(h=e(p.N, BF), gu=e(2 * p.N, BF), h32=e(p.N, F32), q=e(2 * p.N, U8), s=e(p.N // 16, U8), h0=e(p.N, BF),
                dx=e(p.K, BF), dx32=e(p.K, F32))


def test_other_stream_and_repeat():
    p = problem("tall", seed=51)
    assert min(chosen("tall")) > 0
    x, w, dh = p.dev("x", "w", "dh")
    a, b, c = _outputs(p), _outputs(p), _outputs(p)
    _step(p, x, w, dh, a)
    _step(p, x, w, dh, b)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        _step(p, x, w, dh, c)
    st.synchronize()
    for k in a:
        assert torch.equal(a[k], b[k]) and torch.equal(a[k], c[k]), k
    assert torch.equal(a["h"], a["h0"])


def test_graph_replays():
    p = problem("tall", seed=61)
    assert min(chosen("tall")) > 0
    x, w, dh = p.dev("x", "w", "dh")
    o = _outputs(p)
    _step(p, x, w, dh, o)
    torch.cuda.synchronize()
    eager = {k: v.clone() for k, v in o.items()}
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        _step(p, x, w, dh, o)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            _step(p, x, w, dh, o)
    torch.cuda.synchronize()
    for rep in range(3):
        for v in o.values():
            v.zero_()
        if rep == 1:
            _step(p, x, w, dh, o)
        junk = (torch.randn(1 << 20, device=DEV) * 3).sum()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.isfinite(junk)
        for k, v in o.items():
            assert torch.equal(v, eager[k]), (rep, k)


def bf16_64(v):
    """v (float64) rounded to bf16, half to even: 8 significant bits (no overflow or subnormal in these tests)."""
    m, e = np.frexp(v)
    return np.ldexp(np.rint(m * 256) / 256, e)


@pytest.mark.parametrize("shape", [T.SHAPES[6], FORMS["tall"][:4]], ids=["small", "load_waves"])
def test_operand_rounding_is_the_only_one_before_the_result(shape):
    """dx and dw of fp32 against the gradients of a dP rounded to bf16 in 64 bits."""
    p = T.Problem(*shape, seed=5)
    dh, w, x, gu = p.dev("dh", "w", "x", "gu")
    dx, dw = gmm.gmm_bf16_swiglu_bwd(dh, w, p.gs, lhs=x, gu=gu, dx_dtype=F32, dw_dtype=F32)
    d = T.grad64(p, T.f64(p.gu))
    w64, x64 = T.f64(p.w), T.f64(p.x)[:p.used]
    errs = []
    for e in (bf16_64(d), d):
        rdx, rdw = np.zeros((p.M, p.K)), np.zeros((p.G, p.K, 2 * p.N))
        for g, r in p.groups():
            rdx[r], rdw[g] = e[r] @ w64[g].T, x64[r].T @ e[r]
        errs.append([np.linalg.norm(T.f64(a) - b) / np.linalg.norm(b) for a, b in ((dx, rdx), (dw, rdw))])
    assert max(errs[0]) <= 2.0 ** -10, errs
    # a rounding that is spread evenly over half a step: about sqrt(1/3) 2^-8 x 0.75, never above 2^-8
    assert max(errs[1]) <= 2.0 ** -8, errs
