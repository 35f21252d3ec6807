"""GPU: the order of the slots by expert, and rows moved into it and back,
against numpy in 64 bits.

Bounds (u = 2^-24, half a step of fp32).  Orders and moved rows are exact.  A
combined value adds k products and a residual in fp32: (k + 2) u of the sum of
their magnitudes, and half a step of the output's type.  dy is one product:
u and half a step.  dweights adds K products, at most K / 64 + 32 of them or of
partial sums in a row: that many u of the sum of their magnitudes.
"""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_gmm_amd as gmm
import moe_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
U = 2.0 ** -24


def n64(t):
    return t.double().cpu().numpy()


def make_ids(T, k, E, seed, off=0.0, skew=False):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, E, (T, k), generator=g)
    if skew:
        ids = (torch.rand(T, k, generator=g) ** 4 * E).long()
    if off:
        ids[torch.rand(T, k, generator=g) < off] = -1
    return ids.to(I32)


def check_order(ids, G, first=0, rows=None):
    ws = torch.full((gmm.workspace_bytes(gmm.OP_SORT_TOKENS, ids.numel(), 0, 0, G),), 0xA5, dtype=torch.uint8, device=DEV)
    got = gmm.gmm_sort_tokens(ids.to(DEV), G, first=first, rows=rows, ws=ws)
    status = gmm.device_status(ws)
    want = ref.order(ids.numpy(), G, first, rows)
    for a, b in zip(got, want):
        assert a.dtype == I32 and np.array_equal(a.cpu().numpy(), b)
    here = int(((ids >= first) & (ids < first + G)).sum())
    assert status == (gmm.DEV_SUM_GT_M if rows is not None and here > rows else 0)
    return got


# one workgroup; two launches; three launches; each with few and with many experts
@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 256), (5, 3, 7), (64, 1, 2), (100, 6, 60), (512, 8, 256), (500, 8, 257),
                                   (511, 8, 1024), (300, 2, 1025), (513, 8, 256), (1777, 6, 52), (3000, 7, 4096),
                                   (8192, 8, 256), (9000, 8, 128), (8191, 9, 1000), (12345, 7, 4096), (65536, 8, 256),
                                   (300000, 5, 3)])
def test_order(T, k, E):
    check_order(make_ids(T, k, E, T + E), E)
    check_order(make_ids(T, k, E, T + E + 1, off=0.3, skew=True), E)


@pytest.mark.parametrize("T,k,E,first,G", [(50, 4, 64, 48, 16), (2000, 6, 52, 13, 13), (9000, 8, 256, 224, 32), (700, 3, 9, 0, 4),
                                           (40, 2, 5, 5, 3)])
def test_order_of_a_rank(T, k, E, first, G):
    ids = make_ids(T, k, E, T)
    here = int(((ids >= first) & (ids < first + G)).sum())
    for rows in (None, here, here + 17, max(here - 5, 0), here // 3, 0, T * k + 100):
        check_order(ids, G, first, rows)


def test_order_of_odd_ids():
    """Ids far outside the experts, one expert for all, none for any."""
    i32 = torch.iinfo(I32)
    ids = make_ids(400, 4, 16, 3)
    ids[::3, 1], ids[1::3, 2], ids[2::3, 0] = i32.min, i32.max, 16
    check_order(ids, 16)
    check_order(ids, 8, 8)
    check_order(ids, 4, i32.max - 2000)
    for fill in (-1, 0, 15):
        check_order(torch.full((1500, 4), fill, dtype=I32), 16)


def test_order_of_no_tokens():
    for G in (4, 2000):
        for rows in (None, 5):
            check_order(torch.zeros((0, 3), dtype=I32), G, 0, rows)


def plan(T, k, E, seed, rows=None, first=0, G=None, off=0.1):
    G = E if G is None else G
    return check_order(make_ids(T, k, E, seed, off), G, first, rows)


SIZES = [(1, 8, 64, 2048), (1, 1, 1, 8), (37, 3, 5, 72), (300, 6, 60, 1088), (129, 8, 256, 512), (65, 64, 64, 128), (200, 2, 16, 8200)]


def rnd(shape, dt, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dt)


@pytest.mark.parametrize("T,k,E,K", SIZES)
@pytest.mark.parametrize("dt", [BF, F32])
def test_there_and_back(T, k, E, K, dt):
    gs, row_of, slot_of = plan(T, k, E, 7)
    used, M = int(gs.sum()), T * k
    x = rnd((T, K), dt, 1)
    rows = gmm.gmm_dispatch(x.to(DEV), row_of, slot_of)
    assert rows.dtype == dt and np.array_equal(n64(rows), ref.dispatch(n64(x), slot_of.cpu().numpy(), k))
    y = rnd((M, K), dt, 2)
    y[used:] = float("nan")
    w = rnd((T, k), F32, 3)
    w[(row_of == -1).cpu()] = float("nan")          # of slots without a row: never looked at
    for out_dt in (BF, F32):
        for weights, residual in ((None, None), (w, None), (w, rnd((T, K), out_dt, 4)), (None, rnd((T, K), out_dt, 5))):
            got = gmm.gmm_combine(y.to(DEV), row_of, weights=None if weights is None else weights.to(DEV),
                                  residual=None if residual is None else residual.to(DEV), out_dtype=out_dt)
            want, mag = ref.combine(n64(y), row_of.cpu().numpy(), None if weights is None else n64(weights),
                                    None if residual is None else n64(residual))
            assert got.dtype == out_dt
            assert np.all(np.abs(n64(got) - want) <= (k + 2) * U * mag + torch.finfo(out_dt).eps / 2 * np.abs(want))


@pytest.mark.parametrize("T,k,E,K", SIZES)
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("ydt", [BF, F32])
def test_back_and_there(T, k, E, K, dt, ydt):
    gs, row_of, slot_of = plan(T, k, E, 8, rows=T * k + 3)
    used, M = int(gs.sum()), T * k + 3
    dout, y, w = rnd((T, K), dt, 1), rnd((M, K), ydt, 2), rnd((T, k), F32, 3)
    y[used:] = float("nan")
    w[(row_of == -1).cpu()] = float("nan")
    dy, dw = gmm.gmm_combine_bwd(dout.to(DEV), y.to(DEV), row_of, slot_of, w.to(DEV))
    rn = row_of.cpu().numpy()
    rdy, rdw, mag = ref.combine_bwd(n64(dout), n64(y), rn, n64(w), M)
    assert dy.dtype == ydt and dw.dtype == F32
    assert np.all(np.abs(n64(dy) - rdy) <= (torch.finfo(ydt).eps / 2 + U) * np.abs(rdy) + 2.0 ** -126)
    assert np.all(np.abs(n64(dw) - rdw) <= (K / 64 + 32) * U * mag)
    # either alone gives the same
    only, none = gmm.gmm_combine_bwd(dout.to(DEV), None, row_of, slot_of, w.to(DEV), want_dweights=False, dy_dtype=ydt)
    assert none is None and torch.equal(only, dy)
    none, only = gmm.gmm_combine_bwd(dout.to(DEV), y.to(DEV), row_of, slot_of, None, want_dy=False)
    assert none is None and torch.equal(only, dw)


def test_gradients_against_differences():
    """dx of dispatch and (dy, dweights) of combine, by inner products: <f'(v), g> = <v, f'*(g)> for linear maps, exact in
    fp32 for small integers."""
    T, k, E, K = 41, 4, 9, 64
    gs, row_of, slot_of = plan(T, k, E, 9, rows=T * k)
    g = torch.Generator().manual_seed(1)
    ints = lambda *s: torch.randint(-3, 4, s, generator=g).float().to(DEV)
    x, dr, w, y, d = ints(T, K), ints(T * k, K), ints(T, k), ints(T * k, K), ints(T, K)
    used = int(gs.sum())
    dr[used:] = 0
    assert (gmm.gmm_dispatch(x, row_of, slot_of) * dr).sum() == (x * gmm.gmm_combine(dr, row_of)).sum()
    dy, dw = gmm.gmm_combine_bwd(d, y, row_of, slot_of, w)
    base = (gmm.gmm_combine(y, row_of, weights=w) * d).sum()
    assert base == (dy * y).sum() and base == (dw * w).sum()


def test_rows_behind_and_before_stay():
    T, k, E, K = 50, 3, 6, 136
    gs, row_of, slot_of = plan(T, k, E, 10, rows=120)
    big = torch.full((124, K), 7.0, dtype=BF, device=DEV)
    gmm.gmm_dispatch(rnd((T, K), BF, 1).to(DEV), row_of, slot_of, out=big[2:122])
    assert (big[:2] == 7).all() and (big[122:] == 7).all() and (big[2 + int(gs.sum()):122] == 0).all()
    big = torch.full((54, K), 7.0, device=DEV)
    gmm.gmm_combine(rnd((120, K), F32, 2).to(DEV), row_of, out=big[2:52])
    assert (big[:2] == 7).all() and (big[52:] == 7).all()
    assert (big[2:52][(row_of == -1).all(1)] == 0).all()


def test_residual_in_place():
    T, k, E, K = 60, 4, 8, 256
    _, row_of, _ = plan(T, k, E, 11)
    y, r = rnd((T * k, K), BF, 1).to(DEV), rnd((T, K), BF, 2).to(DEV)
    want = gmm.gmm_combine(y, row_of, residual=r)
    assert torch.equal(gmm.gmm_combine(y, row_of, residual=r, out=r), want) and torch.equal(r, want)


def test_bad_rows_are_none():
    """Rows and slots outside the buffers are left out; nothing outside is read or written."""
    T, k, K, M = 20, 3, 64, 40
    row_of = torch.arange(T * k, dtype=I32).reshape(T, k)
    row_of[3, 1], row_of[4, 0], row_of[5, 2] = -5, 2147483647, -2147483648
    slot_of = torch.arange(M, dtype=I32)
    for t, j in ((3, 1), (4, 0), (5, 2)):
        slot_of[t * k + j] = [-5, 2147483647, -2147483648][t - 3]
    x, y, w = rnd((T, K), F32, 1), rnd((M, K), F32, 2), rnd((T, k), F32, 3)
    clean = torch.where((row_of >= 0) & (row_of < M), row_of, torch.full_like(row_of, -1))
    cslot = torch.where((slot_of >= 0) & (slot_of < T * k), slot_of, torch.full_like(slot_of, -1))
    d = lambda *ts: [t.to(DEV) for t in ts]
    rd, sd, cd, csd, xd, yd, wd = d(row_of, slot_of, clean, cslot, x, y, w)
    assert torch.equal(gmm.gmm_dispatch(xd, rd, sd), gmm.gmm_dispatch(xd, cd, csd))
    assert torch.equal(gmm.gmm_combine(yd, rd, weights=wd), gmm.gmm_combine(yd, cd, weights=wd))
    for a, b in zip(gmm.gmm_combine_bwd(xd, yd, rd, sd, wd), gmm.gmm_combine_bwd(xd, yd, cd, csd, wd)):
        assert torch.equal(a, b)
    want, _ = ref.combine(n64(y), clean.numpy(), n64(w))
    assert np.abs(n64(gmm.gmm_combine(yd, rd, weights=wd)) - want).max() < 1e-5


def test_empty_buffers():
    z = lambda *s: torch.zeros(s, dtype=BF, device=DEV)
    r0, s0 = torch.zeros((0, 4), dtype=I32, device=DEV), torch.zeros(0, dtype=I32, device=DEV)
    assert gmm.gmm_dispatch(z(0, 64), r0, s0).shape == (0, 64)
    assert gmm.gmm_combine(z(0, 64), r0).shape == (0, 64)
    none = torch.full((5, 4), -1, dtype=I32, device=DEV)
    res = rnd((5, 64), BF, 1).to(DEV)
    assert torch.equal(gmm.gmm_combine(z(0, 64), none, residual=res), res)
    assert gmm.gmm_dispatch(res, none, s0).shape == (0, 64)
    unowned = torch.full((7,), -1, dtype=I32, device=DEV)
    out = torch.ones((7, 64), dtype=BF, device=DEV)
    assert (gmm.gmm_dispatch(z(0, 64), r0, unowned, out=out) == 0).all()
    dy, dw = gmm.gmm_combine_bwd(res, z(7, 64), none, unowned, torch.ones(5, 4, device=DEV))
    assert (dy == 0).all() and (dw == 0).all()


def test_two_streams_with_workspaces_of_their_own():
    ids = [make_ids(9000, 8, 256, s).to(DEV) for s in (1, 2, 3)]
    want = [gmm.gmm_sort_tokens(i, 256) for i in ids]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ids]
    got = []
    for _ in range(3):
        for i, s in zip(ids, streams):
            with torch.cuda.stream(s):
                got.append(gmm.gmm_sort_tokens(i, 256))
    torch.cuda.synchronize()
    for n, o in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(o, want[n % 3]))


@pytest.mark.parametrize("T,K", [((1 << 20) + 77, 1032), ((1 << 22) + 133, 8)])
def test_more_tokens_than_the_grid(T, K):
    """Workgroups take several tokens one after the other, and runs of slots grow past 1024."""
    if torch.cuda.mem_get_info()[0] < 40e9:
        pytest.skip("needs 40 GB of free device memory")
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    ids = torch.randint(-1, 5, (T, 1), generator=g, device=DEV).to(I32)
    gs, row_of, slot_of = gmm.gmm_sort_tokens(ids, 5)
    order = torch.argsort(torch.where(ids[:, 0] < 0, 5, ids[:, 0].long()), stable=True)
    used = int((ids >= 0).sum())
    assert int(gs.sum()) == used and torch.equal(slot_of[:used].long(), order[:used]) and (slot_of[used:] == -1).all()
    assert torch.equal(row_of[order[:used], 0].long(), torch.arange(used, device=DEV)) and (row_of[ids < 0] == -1).all()
    x = torch.randn(T, K, generator=g, device=DEV, dtype=BF)
    rows = gmm.gmm_dispatch(x, row_of, slot_of)
    assert torch.equal(rows[:used], x[order[:used]]) and not rows[used:].any()
    w = torch.full((T, 1), 0.5, device=DEV)
    back = gmm.gmm_combine(rows, row_of, weights=w)
    assert torch.equal(back, torch.where(ids >= 0, x * 0.5, torch.zeros_like(x)))
    dy, dw = gmm.gmm_combine_bwd(x, rows, row_of, slot_of, w)
    assert torch.equal(dy[:used], x[order[:used]] * 0.5) and not dy[used:].any()
    want = (x.double() ** 2).sum(1)
    assert ((dw[:, 0].double() - torch.where(ids[:, 0] >= 0, want, 0.0)).abs() <= (K / 64 + 32) * U * want).all()


def test_rows_past_32_bits_of_bytes_and_elements():
    """A sorted buffer of more than 2^32 elements: rows at its far end."""
    K, M = 65536, 65600
    y = torch.zeros((M, K), dtype=BF, device=DEV)
    y[M - 3:] = 2.0
    row_of = torch.tensor([[0, M - 1], [M - 2, 5], [M - 3, -1]], dtype=I32, device=DEV)
    w = torch.tensor([[1.0, 0.5], [0.25, 1.0], [2.0, 1.0]], device=DEV)
    out = gmm.gmm_combine(y, row_of, weights=w)
    assert (out[0] == 1).all() and (out[1] == 0.5).all() and (out[2] == 4).all()
    slot_of = torch.full((M,), -1, dtype=I32, device=DEV)
    slot_of[0], slot_of[M - 1], slot_of[M - 2], slot_of[5], slot_of[M - 3] = 0, 1, 2, 3, 4
    x = rnd((3, K), BF, 1).to(DEV)
    rows = gmm.gmm_dispatch(x, row_of, slot_of, out=y)
    assert torch.equal(rows[M - 1], x[0]) and torch.equal(rows[M - 3], x[2]) and torch.equal(rows[M - 2], x[1])
    assert not rows[M - 4].any() and not rows[6].any()
