"""GPU: the router and its gradient against the formulas in 64 bits.

Bounds.  With u = 2^-24 (half a step of fp32) and d the largest |logit - top|
of a case: the difference l - top is off by d u, so exp(l - top) by d u plus
its own rounding (2 u), a sum of E positive terms in lanes of up to 64 and 6
lane moves by 70 u, quotients and products by u each.  A weight is then off by
at most (2 d + 100) u of itself, and a gradient by (4 d + 300) u of the terms it
is made of (a sum of k products more), besides the rounding of what it is
stored as.  Values below the smallest normal number lose bits: 2^-126 is added.
"""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_gmm_amd as gmm
import moe_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
U, TINY = 2.0 ** -24, 2.0 ** -126


def inputs(T, E, dt, seed, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    l = (torch.randn(T, E, generator=g) * spread + torch.randn(E, generator=g) * 0.5).to(dt)
    return l, torch.randn(E, generator=g) * 0.1


def span(l):
    """The largest |logit - top| among experts that are on, and at least 1."""
    c = ref.clean(l)
    with np.errstate(invalid="ignore"):
        d = c.max(axis=1, keepdims=True) - c
    d = np.abs(d[np.isfinite(d)])
    return max(1.0, min(200.0, float(d.max(initial=0)) + float(np.abs(c[np.isfinite(c)]).max(initial=0))))


def check_fwd(l, k, bias, score, normalize, scale):
    b = None if bias is None else bias.to(DEV)
    ids, w = gmm.gmm_route(l.to(DEV), k, bias=b, score=score, normalize=normalize, scale=scale)
    torch.cuda.synchronize()
    ln = l.double().numpy()
    rid, rw = ref.route(ln, k, None if bias is None else bias.double().numpy(), score, normalize, scale)
    assert ids.dtype == torch.int32 and np.array_equal(ids.cpu().numpy(), rid)
    got = w.double().cpu().numpy()
    assert np.all(np.isfinite(got))
    assert np.all(np.abs(got - rw) <= (2 * span(ln) + 100) * U * np.abs(rw) + TINY * abs(scale))
    return ids


def check_bwd(l, ids, score, normalize, scale, out_dtype, seed=5):
    T, k = ids.shape
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(seed))
    got = gmm.gmm_route_bwd(dw.to(DEV), l.to(DEV), ids.to(DEV), score=score, normalize=normalize, scale=scale,
                            out_dtype=out_dtype)
    torch.cuda.synchronize()
    assert got.dtype == (out_dtype or l.dtype)
    ln = l.double().numpy()
    want, mag = ref.route_bwd(dw.double().numpy(), ln, ids.cpu().numpy(), score, normalize, scale)
    half = torch.finfo(got.dtype).eps / 2
    g = got.double().cpu().numpy()
    assert np.all(np.isfinite(g))
    assert np.all(np.abs(g - want) <= (4 * span(ln) + 300) * U * mag + half * np.abs(want) + 4 * TINY * abs(scale))


FORMS = [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)]


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 2, 2), (1, 256, 8), (130, 7, 3), (65, 8, 8), (33, 13, 4), (37, 30, 16),
                                   (203, 60, 6), (64, 64, 64), (19, 65, 8), (41, 255, 7), (500, 256, 8), (9, 257, 10),
                                   (21, 512, 16), (7, 1000, 64), (5, 1025, 8), (3, 4096, 64), (5, 3001, 9)])
@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("bias", [False, True])
def test_choice_weights_and_gradient(T, E, k, dt, bias):
    for i, (score, normalize) in enumerate(FORMS):
        l, b = inputs(T, E, dt, 100 * T + E + i)
        scale = 1.0 if i % 2 else 2.5
        ids = check_fwd(l, k, b if bias else None, score, normalize, scale)
        check_bwd(l, ids, score, normalize, scale, None if i < 2 else (BF if dt == F32 else F32))


# many tokens: four a wave, and from five choices on by sorted lanes
@pytest.mark.parametrize("T,E,k", [(8192, 256, 8), (8195, 250, 16), (8193, 128, 6), (8200, 97, 4), (8192, 130, 5), (8199, 256, 17),
                                   (8192, 65, 9), (9001, 60, 12), (8194, 20, 1)])
@pytest.mark.parametrize("bias", [False, True])
def test_many_tokens(T, E, k, bias):
    for i, (score, normalize) in enumerate(FORMS):
        l, b = inputs(T, E, [F32, BF][i % 2], T + 7 * E + i)     # bf16: many equal logits
        l[::7, E // 2] = float("-inf")
        l[5] = float("-inf")
        ids = check_fwd(l, k, b if bias else None, score, normalize, 1.0)
        if T < 8200:
            check_bwd(l[:300], ids[:300].clone(), score, normalize, 1.0, None)
        # the gradient of many tokens is that of few
        dw = torch.randn(T, k, device=DEV)
        whole = gmm.gmm_route_bwd(dw, l.to(DEV), ids, score=score, normalize=normalize, out_dtype=F32)
        part = gmm.gmm_route_bwd(dw[-1000:].clone(), l[-1000:].to(DEV), ids[-1000:].clone(), score=score, normalize=normalize,
                                 out_dtype=F32)
        tol = (8 * span(l.double().numpy()) + 600) * U * dw[-1000:].abs().max()
        assert ((whole[-1000:] - part).abs() <= tol).all()


@pytest.mark.parametrize("T,E,k", [(8192, 256, 8), (8192, 128, 7), (8192, 256, 16), (70, 256, 8)])
@pytest.mark.parametrize("levels", [1, 2, 5])
def test_equal_keys_of_many_tokens(T, E, k, levels):
    """Few different logits: most choices are the same key, many of the same lane."""
    l = torch.randint(0, levels, (T, E), generator=torch.Generator().manual_seed(E + levels)).float()
    check_fwd(l, k, None, "softmax", True, 1.0)
    check_fwd(l.to(BF), k, torch.zeros(E), "sigmoid", True, 1.0)
    l[:, 3:] = float("-inf")
    ids = check_fwd(l, k, None, "softmax", True, 1.0)
    assert (ids[:, 3:] == -1).all()


@pytest.mark.parametrize("score,normalize", FORMS)
@pytest.mark.parametrize("E", [8, 60, 256, 700])
def test_equal_keys_go_to_the_lower_index(score, normalize, E):
    l = torch.randint(-2, 3, (77, E), generator=torch.Generator().manual_seed(E)).float() * 0.5
    l[5] = 0.0
    l[6, ::2] = -0.0                       # one zero
    for dt in (F32, BF):
        check_fwd(l.to(dt), min(8, E), None, score, normalize, 1.0)
        check_fwd(l.to(dt), min(8, E), torch.zeros(E), score, normalize, 1.0)


@pytest.mark.parametrize("score,normalize", FORMS)
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("E", [8, 60, 256, 300])
def test_experts_that_are_off(score, normalize, bias, E):
    """-infinity and NaN switch an expert off; a token with fewer than k others, or none, gets -1."""
    l, b = inputs(40, E, F32, E)
    l[:, 1] = float("-inf")
    l[:, 3] = float("nan")
    l[4] = float("-inf")
    l[5] = float("nan")
    l[6, 5:] = float("-inf")
    l[7, 2] = torch.finfo(F32).min        # the lowest value of the type is a logit like any other
    l[8] = torch.finfo(F32).min
    k = 6
    ids = check_fwd(l, k, b if bias else None, score, normalize, 1.5)
    off = ((ids == 1) | (ids == 3)).any(1)
    off[8] = False                        # every expert of token 8 is on
    assert (ids[4:6] == -1).all() and not off.any() and (ids[6] == -1).sum() == 3
    check_bwd(l, ids, score, normalize, 1.5, None)
    g = gmm.gmm_route_bwd(torch.ones(40, k, device=DEV), l.to(DEV), ids, score=score, normalize=normalize)
    assert (g[4:6] == 0).all() and (g[:8, [1, 3]] == 0).all() and (g[9:, [1, 3]] == 0).all()


@pytest.mark.parametrize("score,normalize", FORMS)
def test_far_logits(score, normalize):
    """Infinities, and logits whose exponentials overflow or vanish: shares of the chosen scores still add up."""
    l, b = inputs(12, 64, F32, 9)
    l[0, 10] = float("inf")
    l[1] -= 500.0
    l[2] += 500.0
    l[3, :32] -= 90.0
    l[4] *= 60.0
    l[5, 3] = 3e38
    l[6, 3], l[6, 9] = float("inf"), float("inf")
    for bias in (None, b):
        ids = check_fwd(l, 8, bias, score, normalize, 1.0)
        check_bwd(l, ids, score, normalize, 1.0, None)
    if normalize:
        w = gmm.gmm_route(l.to(DEV), 8, score=score)[1]
        assert torch.allclose(w.sum(1), torch.ones(12, device=DEV), atol=1e-5)


def test_bias_chooses_and_does_not_weigh():
    l, _ = inputs(50, 32, F32, 21)
    b = torch.zeros(32)
    b[7], b[11], b[13], b[15] = 100.0, float("-inf"), float("nan"), float("inf")
    ids = check_fwd(l, 4, b, "sigmoid", True, 1.0)
    assert (ids[:, 0] == 15).all() and (ids[:, 1] == 7).all() and not ((ids == 11) | (ids == 13)).any()
    # a bias that takes every expert but two away
    b[:] = float("-inf")
    b[3] = b[9] = 0.0
    ids = check_fwd(l, 4, b, "softmax", True, 1.0)
    assert (ids[:, 2:] == -1).all()


def test_choice_between_scores_that_32_bits_cannot_tell_apart():
    """Keys whose 64-bit values differ below fp32's resolution."""
    E = 64
    l = torch.full((4, E), 3.0)
    l[:, 17] = torch.nextafter(torch.tensor(3.0), torch.tensor(4.0))
    l[1] += 12.0
    check_fwd(l, 3, torch.full((E,), 0.25), "sigmoid", True, 1.0)
    check_fwd(l, 3, torch.full((E,), 0.25), "softmax", True, 1.0)


@pytest.mark.parametrize("T,E,k", [(40, 256, 8), (8192, 256, 8), (8192, 128, 4), (50, 60, 6), (20, 700, 9), (8192, 256, 1)])
def test_ties_at_the_edge_of_the_choice(T, E, k):
    """Keys with a bias around the last chosen one: equal logits and biases (the same key), equal keys of different
    logits and biases, and keys that only 64 bits tell apart, among experts on both sides of the edge."""
    g = torch.Generator().manual_seed(T + E + k)
    l = torch.randint(-3, 4, (T, E), generator=g).float() * 0.5
    for score in ("sigmoid", "softmax"):
        for b in (torch.zeros(E), torch.randint(0, 3, (E,), generator=g).float() * 0.125,
                  torch.where(torch.rand(E, generator=g) < 0.5, 0.0, 2.0 ** -24), torch.full((E,), 2.0 ** 20)):
            check_fwd(l, k, b, score, True, 1.0)
            check_fwd(l.to(BF), k, b, score, False, 1.0)
    near = l + torch.randint(-1, 2, (T, E), generator=g).float() * 2.0 ** -22      # next to each other
    check_fwd(near, k, torch.zeros(E), "sigmoid", True, 1.0)
    check_fwd(near, k, torch.zeros(E), "softmax", True, 1.0)


def test_gradient_of_bad_and_repeated_ids():
    """Ids outside the experts take no part; an expert named twice gets both gradients."""
    l, _ = inputs(6, 40, F32, 31)
    ids = torch.tensor([[0, 1, 2], [-1, 5, 40], [-2147483648, 2147483647, 7], [9, 9, 9], [3, 4, 3], [-1, -1, -1]],
                       dtype=torch.int32)
    for score, normalize in FORMS:
        if normalize:
            continue
        check_bwd(l, ids, score, normalize, 1.0, None)
    for score in ("softmax", "sigmoid"):
        clean_ids = torch.where((ids >= 0) & (ids < 40), ids, torch.full_like(ids, -1))
        check_bwd(l, clean_ids, score, True, 1.0, None)
        dw = torch.randn(6, 3, device=DEV)
        a = gmm.gmm_route_bwd(dw, l.to(DEV), ids.to(DEV), score=score)
        assert torch.equal(a, gmm.gmm_route_bwd(dw, l.to(DEV), clean_ids.to(DEV), score=score))
        for E, many in ((8, 1), (40, 1), (200, 1), (200, 2000), (600, 1), (2000, 1)):
            # the same few experts at every width, for few tokens and for many
            wide = torch.cat([l, torch.full((6, 2000), float("-inf"))], 1)[:, :E].repeat(many, 1)
            i = torch.where(clean_ids < E, clean_ids, torch.full_like(ids, -1)).repeat(many, 1)
            check_bwd(wide[:12], i[:12], score, False, 1.0, None)
            d = dw.repeat(many, 1)
            g = gmm.gmm_route_bwd(d, wide.to(DEV), i.to(DEV), score=score)
            assert torch.equal(g[:6], g[-6:]) and torch.equal(g, gmm.gmm_route_bwd(d, wide.to(DEV), i.to(DEV), score=score))


@pytest.mark.parametrize("score,normalize", FORMS)
def test_gradient_against_differences(score, normalize):
    """Central differences of the 64-bit weights: the gradient is that of what the forward computes."""
    l, b = inputs(5, 24, F32, 41, spread=1.0)
    ids, _ = gmm.gmm_route(l.to(DEV), 4, bias=b.to(DEV), score=score, normalize=normalize, scale=2.0)
    dw = torch.randn(5, 4, generator=torch.Generator().manual_seed(3))
    g = gmm.gmm_route_bwd(dw.to(DEV), l.to(DEV), ids, score=score, normalize=normalize, scale=2.0).double().cpu().numpy()
    idn, ln, h = ids.cpu().numpy(), l.double().numpy(), 1e-5

    def value(z):
        s = ref.share(z, idn, score) if normalize else np.take_along_axis(ref.scores(z, score), idn, 1)
        return (2.0 * s * dw.double().numpy()).sum(axis=1)

    for e in range(24):
        up, down = ln.copy(), ln.copy()
        up[:, e] += h
        down[:, e] -= h
        # fp32 gradient (400 u of terms up to 2 |dw| < 10) and h^2 of third derivatives
        assert np.all(np.abs((value(up) - value(down)) / (2 * h) - g[:, e]) <= 400 * U * 10 + 1e-7)


def test_outputs_given_and_rows_left_alone():
    l, _ = inputs(70, 60, BF, 51)
    ids = torch.full((72, 6), -7, dtype=torch.int32, device=DEV)
    w = torch.full((72, 6), -7.0, device=DEV)
    a, b = gmm.gmm_route(l.to(DEV), 6)
    gmm.gmm_route(l.to(DEV), 6, ids=ids[:70], weights=w[:70])
    assert torch.equal(ids[:70], a) and torch.equal(w[:70], b) and (ids[70:] == -7).all() and (w[70:] == -7).all()
    dl = torch.full((72, 60), -7.0, device=DEV)
    gmm.gmm_route_bwd(torch.ones(70, 6, device=DEV), l.to(DEV), a, out=dl[:70])
    assert (dl[70:] == -7).all() and not (dl[:70] == -7).any()


@pytest.mark.parametrize("T,E,k,dt", [((1 << 22) + 5, 300, 3, BF), ((1 << 24) + 37, 8, 2, BF), ((1 << 24) + 9, 65, 5, BF)])
def test_more_tokens_than_the_grid(T, E, k, dt):
    """Workgroups take several tokens one after the other: the last tokens are those of a call of their own."""
    if torch.cuda.mem_get_info()[0] < 60e9:
        pytest.skip("needs 60 GB of free device memory")
    l = torch.randn(T, E, device=DEV, dtype=dt)
    l[-9000:] = torch.randn(9000, E, generator=torch.Generator().manual_seed(1)).to(DEV, dt)
    b = torch.randn(E, device=DEV) * 0.1
    for how in (dict(normalize=False), dict(bias=b, score="sigmoid")):
        ids, w = gmm.gmm_route(l, k, **how)
        few = gmm.gmm_route(l[-9000:].clone(), k, **how)
        assert torch.equal(ids[-9000:], few[0]) and torch.equal(w[-9000:], few[1])
        how.pop("bias", None)
        dw = torch.ones(T, k, device=DEV)
        dw[-9000:] = torch.randn(9000, k, device=DEV)
        g = gmm.gmm_route_bwd(dw, l, ids, **how)
        assert torch.equal(g[-9000:], gmm.gmm_route_bwd(dw[-9000:].clone(), l[-9000:].clone(), ids[-9000:].clone(), **how))


def test_gradient_of_no_choice_is_not_looked_at():
    l, _ = inputs(9000, 40, F32, 71)
    l[::3] = float("-inf")
    for score, normalize in FORMS:
        for T in (30, 9000):
            ids, _ = gmm.gmm_route(l[:T].to(DEV), 4, score=score, normalize=normalize)
            dw = torch.ones(T, 4, device=DEV)
            dw[ids < 0] = float("nan")
            g = gmm.gmm_route_bwd(dw, l[:T].to(DEV), ids, score=score, normalize=normalize)
            assert torch.isfinite(g).all() and (g[::3] == 0).all()


def test_no_tokens():
    ids, w = gmm.gmm_route(torch.zeros(0, 16, device=DEV), 4)
    assert ids.shape == (0, 4) and w.shape == (0, 4)
    assert gmm.gmm_route_bwd(w, torch.zeros(0, 16, device=DEV), ids).shape == (0, 16)


def test_other_streams_and_repeats():
    l, b = inputs(3000, 256, F32, 61)
    ld, bd = l.to(DEV), b.to(DEV)
    want = gmm.gmm_route(ld, 8, bias=bd, score="sigmoid")
    dw = torch.randn(3000, 8, device=DEV)
    gwant = gmm.gmm_route_bwd(dw, ld, want[0], score="sigmoid")
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            o = gmm.gmm_route(ld, 8, bias=bd, score="sigmoid")
            got.append(o + (gmm.gmm_route_bwd(dw, ld, o[0], score="sigmoid"),))
    torch.cuda.synchronize()
    for o in got:
        assert torch.equal(o[0], want[0]) and torch.equal(o[1], want[1]) and torch.equal(o[2], gwant)
