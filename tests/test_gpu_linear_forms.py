"""GPU: every kernel that the grouped product with an epilogue can run, at sizes
that reach it (checked first), against float64 on the same GPU.  Bounds as in
test_gpu_linear."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_gmm_amd as gmm
from test_gpu_linear import ACTS, TINY, U, half, spread

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, I32, F64 = torch.bfloat16, torch.float32, torch.int32, torch.float64

# name: M, G, K, N, and what gmm_get_tile_config says: kernel, waves, rows, columns
FORMS = {
    "few_narrow": (24, 3, 192, 64, 1, 8, 16, 32),
    "few_wide": (100, 20, 192, 1024, 1, 4, 16, 64),
    "few_32": (500, 5, 448, 320, 1, 4, 32, 64),
    "tiles_128": (3800, 40, 128, 1344, 2, 4, 128, 128),
    "tiles_256": (3800, 40, 320, 1344, 2, 4, 128, 256),
    "tiles_256_odd": (9000, 50, 832, 1728, 2, 4, 128, 256),
    "load_64": (3200, 32, 768, 768, 3, 12, 64, 256),
    "load_96": (4096, 32, 1024, 1024, 3, 12, 96, 256),
    "load_160": (8192, 32, 768, 1024, 3, 12, 160, 256),
    "load_128": (7400, 64, 768, 1024, 3, 12, 128, 256),
    "load_rounds_short": (16500, 64, 512, 2048, 3, 12, 160, 256),
    "load_rounds_160": (16500, 64, 2048, 1024, 3, 12, 160, 256),
    "load_odd": (2300, 16, 832, 832, 3, 12, 64, 256),
}


def chosen(name):
    M, G, K, N = FORMS[name][:4]
    c = gmm.get_tile_config(gmm.OP_BF16_LINEAR, M, K, N, G)
    return c["kernel"], c["waves"], c["tile_m"], c["tile_n"]


def rnd(shape, dt, seed, scale=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dt)


def act64(name, z):
    if name == "relu":
        return z.clamp(min=0), torch.zeros_like(z)
    if name == "silu":
        return z / (1 + torch.exp(-z)), z.abs()
    if name == "gelu":
        return 0.5 * z * torch.special.erfc(-z / 2 ** 0.5), z * z
    if name == "gelu_tanh":
        c = 1.6 * z.abs() * (1 + 0.0447 * z * z)
        return z / (1 + torch.exp(-2 * (2 / np.pi) ** 0.5 * (z + 0.044715 * z ** 3))), c
    return z, torch.zeros_like(z)


def check(M, G, K, N, sizes, act, bias_dt, residual, keep, out_dt, seed):
    x, w = rnd((M, K), BF, seed), rnd((G, K, N), BF, seed + 1, K ** -0.5)
    used = int(np.sum(sizes))
    x[used:] = float("nan")
    b = None if bias_dt is None else rnd((G, N), bias_dt, seed + 2, 0.5)
    res = None
    if residual:
        res = rnd((M, N), out_dt, seed + 3)
        res[used:] = float("inf")
    pre = torch.full((M, N), 9.0, dtype=BF, device=DEV) if keep else None
    out = gmm.gmm_bf16_linear(x, w, torch.tensor(sizes, dtype=I32, device=DEV), bias=b, activation=act, residual=res,
                              out_dtype=out_dt, pre=pre)
    assert not out[used:].any() and (pre is None or not pre[used:].any())
    lo = 0
    for g, s in enumerate(int(v) for v in sizes):
        r = slice(lo, lo + s)
        lo += s
        if s == 0:
            continue
        bg = torch.zeros(N, dtype=F64, device=DEV) if b is None else b[g].to(F64)
        xd, wd = x[r].to(F64), w[g].to(F64)
        z = xd @ wd + bg
        ez = (K + 2) * U * (xd.abs() @ wd.abs() + bg.abs())
        if keep:
            assert ((pre[r].to(F64) - z).abs() <= ez + half(BF) * (z.abs() + ez) + TINY).all(), "pre, group %d" % g
        v, c = act64(act, z)
        rd = torch.zeros_like(v) if res is None else res[r].to(F64)
        e = 1.13 * ez + (16 + 8 * c.clamp(max=100)) * U * v.abs() + U * (v.abs() + rd.abs()) + TINY * (1 + z.abs())
        want = v + rd
        assert ((out[r].to(F64) - want).abs() <= e + half(out_dt) * (want.abs() + e)).all(), "out, group %d" % g
    return x, w, b, res, out


@pytest.mark.parametrize("name", list(FORMS))
@pytest.mark.parametrize("out_dt", [BF, F32])
def test_form(name, out_dt):
    M, G, K, N = FORMS[name][:4]
    assert chosen(name) == FORMS[name][4:]
    i = list(FORMS).index(name)
    for n, (act, bias_dt, residual, keep) in enumerate([(ACTS[i % 5], BF, True, True), (ACTS[(i + 2) % 5], F32, True, False),
                                                        (ACTS[(i + 3) % 5], None, False, True)]):
        # evenly routed, skewed with empty groups, and with rows that no group owns
        sizes = [spread(M, G, 10 * i + n, empty=e, tail=t) for e, t in ((0.0, 0), (0.3, 0), (0.2, M // 7))][n]
        check(M, G, K, N, sizes, act, bias_dt, residual, keep, out_dt, 100 * i + n)


@pytest.mark.parametrize("name", list(FORMS))
def test_form_with_one_group_or_none(name):
    M, G, K, N = FORMS[name][:4]
    one, none = np.zeros(G, dtype=np.int64), np.zeros(G, dtype=np.int64)
    one[G // 2] = M - 5
    for sizes in (one, none):
        check(M, G, K, N, sizes, "silu", BF, True, True, BF, 7)


@pytest.mark.parametrize("name", list(FORMS))
def test_residual_in_place(name):
    M, G, K, N = FORMS[name][:4]
    sizes = spread(M, G, 3, tail=9)
    x, w, b, res, out = check(M, G, K, N, sizes, "none", BF, True, False, BF, 11)
    gs = torch.tensor(sizes, dtype=I32, device=DEV)
    assert gmm.gmm_bf16_linear(x, w, gs, bias=b, residual=res, out=res) is res and torch.equal(res, out)


@pytest.mark.slow
def test_outputs_past_32_bits():
    """More than 2^32 elements of out, residual and pre, and weights of as many: the last rows and experts."""
    M, K, N, G = 70000, 64, 65536, 3
    if torch.cuda.mem_get_info()[0] < 60e9:
        pytest.skip("needs 60 GB of free device memory")
    x = torch.zeros((M, K), dtype=BF, device=DEV)
    x[-5:] = rnd((5, K), BF, 1)
    w = rnd((G, K, N), BF, 2, 0.1)
    gs = torch.tensor([10, 60000, M - 60012], dtype=I32, device=DEV)   # two rows behind the last group
    b, res = rnd((G, N), BF, 3), torch.zeros((M, N), dtype=BF, device=DEV)
    res[-5:] = rnd((5, N), BF, 4)
    pre = torch.empty((M, N), dtype=BF, device=DEV)
    gmm.gmm_bf16_linear(x, w, gs, bias=b, activation="silu", residual=res, out=res, pre=pre)
    z = x[-5:-2].to(F64) @ w[2].to(F64) + b[2].to(F64)
    assert not res[-2:].any() and not pre[-2:].any()
    assert ((pre[-5:-2].to(F64) - z).abs() <= 1e-4 + half(BF) * z.abs()).all()
    want = z / (1 + torch.exp(-z)) + rnd((5, N), BF, 4)[:3].to(F64)
    assert ((res[-5:-2].to(F64) - want).abs() <= 1e-4 + half(BF) * want.abs()).all()
    assert torch.equal(pre[-6], b[2]) and torch.equal(pre[0], b[0])    # rows of zeros


@pytest.mark.slow
def test_weights_past_32_bits():
    K, N, G, M = 8192, 8192, 66, 96                                    # 4.4e9 weights
    if torch.cuda.mem_get_info()[0] < 40e9:
        pytest.skip("needs 40 GB of free device memory")
    w = torch.zeros((G, K, N), dtype=BF, device=DEV)
    w[G - 1] = rnd((K, N), BF, 1, K ** -0.5)
    x = rnd((M, K), BF, 2)
    gs = torch.zeros(G, dtype=I32, device=DEV)
    gs[0], gs[G - 1] = 32, 64
    out = gmm.gmm_bf16_linear(x, w, gs, out_dtype=F32)
    want = x[32:].to(F64) @ w[G - 1].to(F64)
    assert not out[:32].any()
    assert ((out[32:].to(F64) - want).abs() <= (K + 2) * U * (x[32:].to(F64).abs() @ w[G - 1].to(F64).abs())).all()
