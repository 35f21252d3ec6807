"""GPU: activations of the product with an epilogue at values that are not
ordinary numbers, forward and slope, in every form of the forward.

The value that is stored is the activation of one product: identity weights, so
the sums are the rows of x themselves, exact."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_gmm_amd as gmm
from test_gpu_linear import ACTS
from test_gpu_linear_forms import FORMS, chosen

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
NAN = float("nan")


def eye(N):
    return torch.eye(N, dtype=BF, device=DEV).reshape(1, N, N)


def slopes(pre, act):
    """act'(pre) of each value: dout of ones, db of one row a group."""
    M, N = pre.shape
    one = torch.ones((M, N), dtype=BF, device=DEV)
    w = torch.zeros((M, 64, N), dtype=BF, device=DEV)
    dx, _, db = gmm.gmm_bf16_linear_bwd(one, w, torch.ones(M, dtype=I32, device=DEV), pre=pre, activation=act, want_dw=False)
    return dx, db


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [5, 3000])
@pytest.mark.parametrize("out_dt", [BF, F32])
def test_nan_in_a_used_row_reaches_the_output(act, M, out_dt):
    """Few-row tiles and 128-row tiles: the row is NaN in out and pre, its neighbours are not touched."""
    N = 64 if M == 5 else 1088
    x = torch.randn((M, N), generator=torch.Generator().manual_seed(1)).to(BF)
    x[M // 2, 7] = NAN
    pre = torch.empty((M, N), dtype=BF, device=DEV)
    out = gmm.gmm_bf16_linear(x.to(DEV), eye(N), torch.tensor([M], dtype=I32, device=DEV), activation=act, out_dtype=out_dt,
                              pre=pre)
    nan = torch.zeros((M, N), dtype=torch.bool)
    nan[M // 2] = True                                  # NaN times the weights' zeros
    assert torch.equal(out.isnan().cpu(), nan) and torch.equal(pre.isnan().cpu(), nan)


@pytest.mark.parametrize("name", list(FORMS))
@pytest.mark.parametrize("act", ["relu", "gelu"])
def test_nan_in_every_form(name, act):
    M, G, K, N = FORMS[name][:4]
    assert chosen(name) == FORMS[name][4:]
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn((M, K), generator=g, device=DEV).to(BF)
    w = torch.randn((G, K, N), generator=g, device=DEV).to(BF)
    x[M // 3] = NAN
    gs = torch.full((G,), M // G, dtype=I32, device=DEV)
    gs[0] += M - int(gs.sum())
    out = gmm.gmm_bf16_linear(x, w, gs, activation=act)
    rows = out.isnan().any(1)
    assert out[M // 3].isnan().all() and int(rows.sum()) == 1


def test_relu_of_zeros_and_infinities():
    N = 64
    z = torch.zeros((1, N), dtype=BF)
    z[0, :4] = torch.tensor([-0.0, 0.0, 1e-38, -1e-38])
    pre = torch.tensor([[-0.0, 0.0, float("inf"), -float("inf"), 1e-38, -1e-38] + [2.0] * 58], dtype=BF)
    out = gmm.gmm_bf16_linear(z.to(DEV), eye(N), torch.ones(1, dtype=I32, device=DEV), activation="relu", out_dtype=F32).cpu()
    assert torch.equal(out, z.float().clamp(min=0))
    _, db = slopes(pre.to(DEV), "relu")
    assert torch.equal(db.cpu(), (pre > 0).float())


@pytest.mark.parametrize("act", [a for a in ACTS if a != "none"])
def test_slope_of_nan_is_nan(act):
    N = 64
    pre = torch.zeros((3, N), dtype=BF, device=DEV)
    pre[1, 5] = NAN
    dx, db = slopes(pre, act)
    nan = torch.zeros((3, N), dtype=torch.bool, device=DEV)
    nan[1, 5] = True
    assert torch.equal(db.isnan(), nan)
    assert dx[1].isnan().all() and not dx[0].isnan().any() and not dx[2].isnan().any()


FAR = [2.0 ** 40, 1.5 * 2.0 ** 63, 2.0 ** 64, 2.0 ** 65, 1e25, 3e38]     # squares and cubes past the largest number


@pytest.mark.parametrize("act", [a for a in ACTS if a != "none"])
def test_far_values(act):
    """Far from 0 every activation is max(z, 0) and its slope the step, to the last bit."""
    N = 64
    z = torch.zeros((1, N), dtype=BF)
    z[0, :2 * len(FAR)] = torch.tensor(FAR + [-v for v in FAR]).to(BF)
    out = gmm.gmm_bf16_linear(z.to(DEV), eye(N), torch.ones(1, dtype=I32, device=DEV), activation=act, out_dtype=F32).cpu()
    assert torch.equal(out, z.float().clamp(min=0))
    _, db = slopes(z.to(DEV), act)
    n = 2 * len(FAR)
    assert torch.equal(db.cpu()[:, :n], (z > 0).float()[:, :n])
