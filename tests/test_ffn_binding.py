"""The binding of include/gmm_ffn.h refuses tensors that are not on the GPU of
the call's first operand: a host address that reaches a kernel is an access
fault, not an error.  No call here reaches the library's launch (meta tensors
stand for another device)."""
import pytest
import torch

import moe_grouped_gemm_gmm_amd as gmm
from moe_grouped_gemm_gmm_amd import ffn

BF, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
M, K, N, G = 4, 64, 64, 2


class Lib:
    """Stands for the library: a call that gets this far would have launched."""

    def __getattr__(self, name):
        def call(*args):
            raise AssertionError("%s was called" % name)
        return call


@pytest.fixture(autouse=True)
def no_launch(monkeypatch):
    monkeypatch.setattr(ffn, "load_library", Lib)


def t(shape, dt, dev="cpu"):
    return torch.zeros(shape, dtype=dt, device=dev)


def forward_args():
    return dict(lhs=t((M, K), BF), rhs=t((G, K, 2 * N), BF), group_sizes=t((G,), I32), out=t((M, N), BF),
                gu=t((M, 2 * N), BF), ws=t((256,), U8))


def forward_mx8_args():
    a = forward_args()
    del a["gu"]
    return dict(a, gu_q=t((M, 2 * N), U8), gu_scale=t((M, 2 * N // 32), U8))


def backward_args():
    return dict(dh=t((M, N), BF), rhs=t((G, K, 2 * N), BF), group_sizes=t((G,), I32), lhs=t((M, K), BF),
                gu=t((M, 2 * N), BF), dx=t((M, K), BF), dw=t((G, K, 2 * N), F32), h=t((M, N), BF),
                ws=t((256 + 4 * M * N,), U8))


def backward_mx8_args():
    a = backward_args()
    del a["lhs"], a["gu"]
    return dict(a, lhs_q=t((M, K), U8), lhs_scale=t((M, K // 32), U8), gu_q=t((M, 2 * N), U8),
                gu_scale=t((M, 2 * N // 32), U8))


def quantize_args():
    return dict(x=t((M, K), BF), q=t((M, K), U8), scale=t((M, K // 32), U8))


def dequantize_args():
    return dict(q=t((M, K), U8), scale=t((M, K // 32), U8), out=t((M, K), F32))


def tgmm_args():
    return dict(x_q=t((M, K), U8), x_scale=t((M, K // 32), U8), dy=t((M, N), BF), group_sizes=t((G,), I32),
                out=t((G, K, N), BF), ws=t((256,), U8))


CALLS = [(gmm.gmm_bf16_swiglu, forward_args), (gmm.gmm_bf16_swiglu, forward_mx8_args),
         (gmm.gmm_bf16_swiglu_bwd, backward_args), (gmm.gmm_bf16_swiglu_bwd, backward_mx8_args),
         (gmm.gmm_quantize_mx8, quantize_args), (gmm.gmm_dequantize_mx8, dequantize_args),
         (gmm.tgmm_mx8, tgmm_args)]
ONE = [(f, a, n) for f, a in CALLS for n in list(a())[1:]]


@pytest.mark.parametrize("call,args,name", ONE, ids=["%s-%s" % (a.__name__, n) for _, a, n in ONE])
def test_one_tensor_on_another_device(call, args, name):
    kw = args()
    kw[name] = kw[name].to("meta")
    with pytest.raises(ValueError, match="%s is on meta" % name):
        call(**kw)


@pytest.mark.parametrize("call,args", CALLS, ids=[a.__name__ for _, a in CALLS])
def test_tensors_in_host_memory(call, args):
    with pytest.raises(ValueError, match="not on a GPU"):
        call(**args())


@pytest.mark.parametrize("call,args", CALLS, ids=[a.__name__ for _, a in CALLS])
def test_outputs_are_not_made_in_host_memory(call, args):
    """Without outputs and workspace given, too."""
    kw = {k: v for k, v in args().items() if k not in ("out", "ws", "dx", "dw", "h", "q", "scale") or
          (call is gmm.gmm_dequantize_mx8 and k != "out")}
    with pytest.raises(ValueError, match="not on a GPU"):
        call(**kw)
