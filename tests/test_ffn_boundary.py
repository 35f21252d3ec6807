"""The C ABI of include/gmm_ffn.h on the CPU: exports, workspace sizes and the
refusals of every call, all before any launch (no call here reaches the GPU),
and the binding's own checks of shapes and types."""
import ctypes
import os
import re

import pytest
import torch

import moe_grouped_gemm_gmm_amd as gmm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SHAPE, ALIGN, DTYPE, WORKSPACE = 0, 1, 2, 3, 4, 5
A, MIS = 0x10000, 0x10008      # never dereferenced: the checks fail first
BIG = 1 << 40


def P(x):
    return ctypes.c_void_p(x) if x else None


@pytest.fixture(scope="module")
def lib():
    return gmm.load_library()


def test_exports(lib):
    text = open(os.path.join(ROOT, "include", "gmm_ffn.h")).read()
    names = sorted(set(re.findall(r"GMM_API\s+[\w\s\*]*?\b(\w+)\s*\(", text)))
    assert names == sorted(gmm.FFN_EXPORTS)
    for n in names:
        assert hasattr(lib, n) and hasattr(gmm, n), n


def test_workspace_bytes(lib):
    w = lib.gmm_workspace_bytes
    assert w(gmm.OP_BF16_SWIGLU, 100, 128, 64, 2) == 256
    assert w(gmm.OP_TGMM_MX8, 100, 128, 64, 2) == 256
    assert w(gmm.OP_BF16_SWIGLU_BWD, 100, 128, 64, 2) == 256 + 100 * 2 * 64 * 2
    assert w(gmm.OP_BF16_SWIGLU_BWD, 0, 128, 64, 2) == 256
    # past 32 bits
    assert w(gmm.OP_BF16_SWIGLU_BWD, 1 << 20, 128, 1 << 16, 2) == 256 + (1 << 38)
    assert w(15, 1, 64, 64, 1) == 0 and w(19, 1, 64, 64, 1) == 0


def fwd(lib, lhs=A, rhs=A, gs=A, M=100, K=128, N=192, G=4, out=A, dt=1, gu=0, q=0, s=0, ws=A, wsb=256):
    return lib.gmm_bf16_swiglu(P(lhs), P(rhs), P(gs), M, K, N, G, P(out), dt, P(gu), P(q), P(s), P(ws), wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(lhs=0), NULL), (dict(rhs=0), NULL), (dict(gs=0), NULL), (dict(out=0), NULL),
    (dict(lhs=MIS), ALIGN), (dict(rhs=MIS), ALIGN), (dict(out=MIS), ALIGN), (dict(gu=MIS), ALIGN),
    (dict(q=MIS, s=A), ALIGN), (dict(q=A, s=MIS), ALIGN),
    (dict(q=A), NULL), (dict(s=A), NULL), (dict(gu=A, q=A, s=A), DTYPE), (dict(gu=A, s=A), DTYPE),
    (dict(dt=2), DTYPE), (dict(dt=9), DTYPE),
    (dict(K=96), SHAPE), (dict(K=0), SHAPE), (dict(N=96), SHAPE), (dict(N=-64), SHAPE), (dict(M=-1), SHAPE),
    (dict(G=0), SHAPE), (dict(G=5000), SHAPE), (dict(N=1 << 30), SHAPE), (dict(M=(1 << 31) - 1), SHAPE),
    (dict(M=(1 << 31) - 2048, N=1 << 29), SHAPE),                # grid
    (dict(ws=0), WORKSPACE), (dict(wsb=255), WORKSPACE), (dict(ws=MIS), ALIGN),
    (dict(M=0, lhs=0, out=0), OK), (dict(M=0, ws=0), WORKSPACE), (dict(M=0, rhs=0), NULL),
])
def test_forward_refusals(lib, kw, status):
    assert fwd(lib, **kw) == status
    if status:
        assert lib.gmm_last_error()


def bwd(lib, dh=A, rhs=A, gs=A, x=A, xq=0, xs=0, gu=A, q=0, s=0, M=100, K=128, N=192, G=4, dx=A, dxt=1, dw=A,
        dwt=1, h=0, ws=A, wsb=BIG):
    return lib.gmm_bf16_swiglu_bwd(P(dh), P(rhs), P(gs), P(x), P(xq), P(xs), P(gu), P(q), P(s), M, K, N, G, P(dx),
                                   dxt, P(dw), dwt, P(h), P(ws), wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dh=0), NULL), (dict(rhs=0), NULL), (dict(gs=0), NULL), (dict(x=0), NULL), (dict(gu=0), NULL),
    (dict(x=0, xq=A), NULL), (dict(x=0, xs=A), NULL), (dict(gu=0, q=A), NULL), (dict(gu=0, s=A), NULL),
    (dict(xq=A, xs=A), DTYPE), (dict(q=A, s=A), DTYPE), (dict(xq=A), DTYPE),
    (dict(dx=0, dw=0), NULL),                                   # nothing asked for
    (dict(dxt=2), DTYPE), (dict(dwt=2), DTYPE),
    (dict(dh=MIS), ALIGN), (dict(x=MIS), ALIGN), (dict(x=0, xq=MIS, xs=A), ALIGN), (dict(gu=MIS), ALIGN),
    (dict(gu=0, q=A, s=MIS), ALIGN), (dict(dx=MIS), ALIGN), (dict(dw=MIS), ALIGN), (dict(h=MIS), ALIGN),
    (dict(rhs=MIS), ALIGN), (dict(ws=MIS), ALIGN),
    (dict(K=32), SHAPE), (dict(N=32), SHAPE), (dict(G=0), SHAPE), (dict(M=-5), SHAPE),
    (dict(G=4096, K=1 << 24, N=1 << 24), SHAPE),                # grid of the weight gradient
    (dict(wsb=256 + 100 * 2 * 192 * 2 - 1), WORKSPACE), (dict(ws=0), WORKSPACE),
    (dict(M=0, dh=0, x=0, gu=0, dx=0, dw=0), OK),
])
def test_backward_refusals(lib, kw, status):
    assert bwd(lib, **kw) == status
    if status:
        assert lib.gmm_last_error()


def test_checkpoint_refusals(lib):
    q, d = lib.gmm_quantize_mx8, lib.gmm_dequantize_mx8
    assert q(P(A), 2, 4, 64, P(A), P(A), None) == DTYPE
    assert q(P(A), 1, 4, 40, P(A), P(A), None) == SHAPE
    assert q(P(A), 1, 4, 0, P(A), P(A), None) == SHAPE
    assert q(P(A), 1, -1, 64, P(A), P(A), None) == SHAPE
    assert q(P(A), 1, 1 << 30, 1 << 14, P(A), P(A), None) == SHAPE
    assert q(None, 1, 4, 64, P(A), P(A), None) == NULL
    assert q(P(A), 1, 4, 64, P(MIS), P(A), None) == ALIGN
    assert q(P(A), 1, 4, 64, P(A), P(MIS), None) == ALIGN
    assert q(None, 1, 0, 64, None, None, None) == OK
    assert d(P(A), P(A), 4, 64, P(A), 2, None) == DTYPE
    assert d(P(A), P(A), 4, 16, P(A), 1, None) == SHAPE
    assert d(P(A), None, 4, 64, P(A), 1, None) == NULL
    assert d(P(A), P(A), 4, 64, P(MIS), 1, None) == ALIGN
    assert d(None, None, 0, 64, None, 1, None) == OK


def tg(lib, q=A, s=A, dy=A, gs=A, M=100, K=128, N=192, G=4, dw=A, dt=1, ws=A, wsb=256):
    return lib.tgmm_mx8(P(q), P(s), P(dy), P(gs), M, K, N, G, P(dw), dt, P(ws), wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=0), NULL), (dict(s=0), NULL), (dict(dy=0), NULL), (dict(gs=0), NULL), (dict(dw=0), NULL),
    (dict(q=MIS), ALIGN), (dict(s=MIS), ALIGN), (dict(dy=MIS), ALIGN), (dict(dw=MIS), ALIGN),
    (dict(K=32), SHAPE), (dict(N=100), SHAPE), (dict(G=-1), SHAPE), (dict(M=-1), SHAPE), (dict(dt=2), DTYPE),
    (dict(G=4096, K=1 << 24, N=1 << 24), SHAPE), (dict(ws=0), WORKSPACE), (dict(wsb=100), WORKSPACE),
])
def test_weight_gradient_refusals(lib, kw, status):
    assert tg(lib, **kw) == status
    assert lib.gmm_last_error()


def test_existing_operations_keep_their_ids(lib):
    c = gmm.TileConfig(kernel=1)
    for op in (gmm.OP_BF16_SWIGLU, gmm.OP_BF16_SWIGLU_BWD, gmm.OP_TGMM_MX8):
        assert lib.gmm_set_tile_config(op, ctypes.byref(c)) == SHAPE      # no tile configuration


def test_binding_checks_shapes_and_types():
    bf, f32, u8 = torch.bfloat16, torch.float32, torch.uint8
    x, w = torch.zeros(4, 64, dtype=bf), torch.zeros(2, 64, 128, dtype=bf)
    gs = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        gmm.gmm_bf16_swiglu(x, torch.zeros(2, 128, 128, dtype=bf), gs)
    with pytest.raises(ValueError):
        gmm.gmm_bf16_swiglu(x, w, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(TypeError):
        gmm.gmm_bf16_swiglu(x, w, gs.long())
    with pytest.raises(TypeError):
        gmm.gmm_bf16_swiglu(x.float(), w, gs)
    with pytest.raises(ValueError):
        gmm.gmm_bf16_swiglu(x, w, gs, gu=torch.zeros(4, 64, dtype=bf))
    with pytest.raises(TypeError):
        gmm.gmm_bf16_swiglu(x, w, gs, gu=torch.zeros(4, 128, dtype=f32))
    with pytest.raises(ValueError):
        gmm.gmm_bf16_swiglu(x, w, gs, gu_q=torch.zeros(4, 128, dtype=u8), gu_scale=torch.zeros(4, 2, dtype=u8))
    dh = torch.zeros(4, 64, dtype=bf)
    with pytest.raises(ValueError):
        gmm.gmm_bf16_swiglu_bwd(torch.zeros(4, 128, dtype=bf), w, gs, lhs=x, gu=torch.zeros(4, 128, dtype=bf))
    with pytest.raises(ValueError):
        gmm.gmm_bf16_swiglu_bwd(dh, w, gs, lhs=torch.zeros(3, 64, dtype=bf), gu=torch.zeros(4, 128, dtype=bf))
    with pytest.raises(TypeError):
        gmm.gmm_bf16_swiglu_bwd(dh, w, gs, lhs=x.float(), gu=torch.zeros(4, 128, dtype=bf))
    with pytest.raises(ValueError):
        gmm.tgmm_mx8(torch.zeros(4, 64, dtype=u8), torch.zeros(4, 2, dtype=u8), torch.zeros(5, 64, dtype=bf), gs)
    with pytest.raises(ValueError):
        gmm.tgmm_mx8(torch.zeros(4, 64, dtype=u8), torch.zeros(4, 1, dtype=u8), dh, gs)
    with pytest.raises(ValueError):
        gmm.gmm_dequantize_mx8(torch.zeros(4, 64, dtype=u8), torch.zeros(4, 1, dtype=u8))
    with pytest.raises(TypeError):
        gmm.gmm_quantize_mx8(torch.zeros(4, 64, dtype=torch.float16))
