"""The C ABI of include/gmm_moe.h on the CPU: exports, workspace sizes and the
refusals of every call, all before any launch (no call here reaches the GPU),
and the binding's own checks of shapes, types and devices."""
import ctypes
import os
import re

import pytest
import torch

import moe_grouped_gemm_gmm_amd as gmm
from moe_grouped_gemm_gmm_amd import moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SHAPE, ALIGN, DTYPE, WORKSPACE = 0, 1, 2, 3, 4, 5
A, MIS = 0x10000, 0x10008      # never dereferenced: the checks fail first
BIG = 1 << 40
F32, BF, I32, U8 = torch.float32, torch.bfloat16, torch.int32, torch.uint8


def P(x):
    return ctypes.c_void_p(x) if x else None


@pytest.fixture(scope="module")
def lib():
    return gmm.load_library()


def test_exports(lib):
    text = open(os.path.join(ROOT, "include", "gmm_moe.h")).read()
    names = sorted(set(re.findall(r"GMM_API\s+[\w\s\*]*?\b(\w+)\s*\(", text)))
    assert names == sorted(gmm.MOE_EXPORTS)
    for n in names:
        assert hasattr(lib, n) and hasattr(gmm, n), n


def test_workspace_of_the_order(lib):
    def w(n, G):
        return lib.gmm_workspace_bytes(gmm.OP_SORT_TOKENS, n, 0, 0, G)
    # the status block, and where one workgroup does not take all slots counts of every run of them and their totals
    assert w(8, 256) == 256 and w(4096, 1024) == 256
    assert w(4097, 256) == 256 + 4 * 6 * 256
    assert w(0, 4096) == 256 + 4 * 2 * 4096
    assert w(65536, 256) == 256 + 4 * 65 * 256
    assert w((1 << 31) - 1024, 4096) <= 256 + 4 * 1025 * 4096      # bounded however many slots
    assert w(-5, 2000) == w(0, 2000) and w(100, 0) == 256


def route(lib, l=A, dt=0, b=0, T=10, E=64, k=4, score=0, ids=A, w=A):
    return lib.gmm_route(P(l), dt, P(b), T, E, k, score, 1, 1.0, P(ids), P(w), None)


@pytest.mark.parametrize("kw,status", [
    (dict(l=0), NULL), (dict(ids=0), NULL), (dict(w=0), NULL), (dict(l=MIS), ALIGN), (dict(b=MIS), ALIGN),
    (dict(ids=MIS), ALIGN), (dict(w=MIS), ALIGN), (dict(dt=2), DTYPE), (dict(score=2), DTYPE), (dict(score=-1), DTYPE),
    (dict(E=0), SHAPE), (dict(E=4097), SHAPE), (dict(k=0), SHAPE), (dict(k=65, E=128), SHAPE), (dict(k=5, E=4), SHAPE),
    (dict(T=-1), SHAPE), (dict(T=1 << 30), SHAPE), (dict(T=1 << 40), SHAPE), (dict(T=0, l=0, ids=0, w=0), OK),
])
def test_route_refusals(lib, kw, status):
    assert route(lib, **kw) == status
    if status:
        assert lib.gmm_last_error()


def route_bwd(lib, dw=A, l=A, dt=0, ids=A, T=10, E=64, k=4, score=1, dl=A, ot=0):
    return lib.gmm_route_bwd(P(dw), P(l), dt, P(ids), T, E, k, score, 0, 1.0, P(dl), ot, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dw=0), NULL), (dict(l=0), NULL), (dict(ids=0), NULL), (dict(dl=0), NULL), (dict(dw=MIS), ALIGN),
    (dict(l=MIS), ALIGN), (dict(ids=MIS), ALIGN), (dict(dl=MIS), ALIGN), (dict(dt=2), DTYPE), (dict(ot=2), DTYPE),
    (dict(score=7), DTYPE), (dict(E=-1), SHAPE), (dict(k=100, E=200), SHAPE), (dict(T=-3), SHAPE),
    (dict(T=0, dw=0, l=0, ids=0, dl=0), OK),
])
def test_route_bwd_refusals(lib, kw, status):
    assert route_bwd(lib, **kw) == status


def sort(lib, ids=A, T=10, k=4, first=0, G=16, M=40, gs=A, row=A, slot=A, ws=A, wsb=BIG):
    return lib.gmm_sort_tokens(P(ids), T, k, first, G, M, P(gs), P(row), P(slot), P(ws), wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(ids=0), NULL), (dict(gs=0), NULL), (dict(row=0), NULL), (dict(slot=0), NULL), (dict(ids=MIS), ALIGN),
    (dict(gs=MIS), ALIGN), (dict(row=MIS), ALIGN), (dict(slot=MIS), ALIGN), (dict(ws=MIS), ALIGN),
    (dict(G=0), SHAPE), (dict(G=4097), SHAPE), (dict(M=-1), SHAPE), (dict(M=1 << 31), SHAPE), (dict(first=-1), SHAPE),
    (dict(first=1 << 31), SHAPE), (dict(T=-1), SHAPE), (dict(k=0), SHAPE), (dict(k=65), SHAPE),
    (dict(T=1 << 30, k=2), SHAPE), (dict(ws=0), WORKSPACE), (dict(wsb=255), WORKSPACE),
    (dict(T=2000, wsb=256 + 4 * 9 * 16 - 1), WORKSPACE),
])
def test_order_refusals(lib, kw, status):
    assert sort(lib, **kw) == status


def dispatch(lib, x=A, dt=1, row=A, slot=A, T=10, k=4, M=40, K=64, out=A):
    return lib.gmm_dispatch(P(x), dt, P(row), P(slot), T, k, M, K, P(out), None)


def combine(lib, y=A, yt=1, row=A, w=A, res=A, T=10, k=4, M=40, K=64, out=A, ot=1):
    return lib.gmm_combine(P(y), yt, P(row), P(w), P(res), T, k, M, K, P(out), ot, None)


def combine_bwd(lib, d=A, dt=1, y=A, yt=1, row=A, slot=A, w=A, T=10, k=4, M=40, K=64, dy=A, dw=A):
    return lib.gmm_combine_bwd(P(d), dt, P(y), yt, P(row), P(slot), P(w), T, k, M, K, P(dy), P(dw), None)


SIZES = [(dict(K=4), SHAPE), (dict(K=0), SHAPE), (dict(K=100), SHAPE), (dict(K=-8), SHAPE), (dict(k=0), SHAPE),
         (dict(k=65), SHAPE), (dict(T=-1), SHAPE), (dict(M=-1), SHAPE), (dict(M=1 << 31), SHAPE), (dict(T=1 << 31), SHAPE)]


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(x=0), NULL), (dict(row=0), NULL), (dict(slot=0), NULL), (dict(out=0), NULL), (dict(x=MIS), ALIGN),
    (dict(row=MIS), ALIGN), (dict(slot=MIS), ALIGN), (dict(out=MIS), ALIGN), (dict(dt=2), DTYPE),
    (dict(M=0, slot=0, out=0), OK),
])
def test_dispatch_refusals(lib, kw, status):
    assert dispatch(lib, **kw) == status


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(y=0), NULL), (dict(row=0), NULL), (dict(out=0), NULL), (dict(y=MIS), ALIGN), (dict(row=MIS), ALIGN),
    (dict(w=MIS), ALIGN), (dict(res=MIS), ALIGN), (dict(out=MIS), ALIGN), (dict(yt=2), DTYPE), (dict(ot=2), DTYPE),
    (dict(T=0, row=0, out=0), OK),
])
def test_combine_refusals(lib, kw, status):
    assert combine(lib, **kw) == status


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(d=0), NULL), (dict(row=0), NULL), (dict(slot=0), NULL), (dict(w=0), NULL), (dict(y=0), NULL),
    (dict(dy=0, dw=0), NULL), (dict(d=MIS), ALIGN), (dict(y=MIS), ALIGN), (dict(row=MIS), ALIGN), (dict(slot=MIS), ALIGN),
    (dict(w=MIS), ALIGN), (dict(dy=MIS), ALIGN), (dict(dw=MIS), ALIGN), (dict(dt=2), DTYPE), (dict(yt=2), DTYPE),
    (dict(yt=-1), DTYPE), (dict(T=0, M=0, d=0, row=0, slot=0, w=0, y=0, dy=0, dw=0), OK),
])
def test_combine_bwd_refusals(lib, kw, status):
    assert combine_bwd(lib, **kw) == status


def linear(lib, x=A, w=A, gs=A, M=100, K=128, N=192, G=4, b=A, bt=1, act=3, res=A, out=A, ot=1, pre=A, ws=A, wsb=256):
    return lib.gmm_bf16_linear(P(x), P(w), P(gs), M, K, N, G, P(b), bt, act, P(res), P(out), ot, P(pre), P(ws), wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=0), NULL), (dict(w=0), NULL), (dict(gs=0), NULL), (dict(out=0), NULL),
    (dict(x=MIS), ALIGN), (dict(w=MIS), ALIGN), (dict(b=MIS), ALIGN), (dict(res=MIS), ALIGN), (dict(out=MIS), ALIGN),
    (dict(pre=MIS), ALIGN), (dict(ws=MIS), ALIGN), (dict(bt=2), DTYPE), (dict(ot=2), DTYPE), (dict(act=5), DTYPE),
    (dict(act=-1), DTYPE), (dict(K=96), SHAPE), (dict(K=0), SHAPE), (dict(N=96), SHAPE), (dict(N=-64), SHAPE),
    (dict(M=-1), SHAPE), (dict(G=0), SHAPE), (dict(G=4097), SHAPE), (dict(M=(1 << 31) - 1), SHAPE),
    (dict(M=(1 << 31) - 2048, N=1 << 29), SHAPE),                # grid
    (dict(ws=0), WORKSPACE), (dict(wsb=255), WORKSPACE),
    (dict(M=0, x=0, out=0, b=0, res=0, pre=0), OK), (dict(M=0, ws=0), WORKSPACE), (dict(M=0, w=0), NULL),
])
def test_linear_refusals(lib, kw, status):
    assert linear(lib, **kw) == status
    if status:
        assert lib.gmm_last_error()


def linear_bwd(lib, d=A, w=A, gs=A, x=A, pre=A, act=3, M=100, K=128, N=192, G=4, dx=A, dxt=1, dw=A, dwt=1, db=A, dbt=0,
               ws=A, wsb=BIG):
    return lib.gmm_bf16_linear_bwd(P(d), P(w), P(gs), P(x), P(pre), act, M, K, N, G, P(dx), dxt, P(dw), dwt, P(db), dbt,
                                   P(ws), wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(d=0), NULL), (dict(w=0), NULL), (dict(gs=0), NULL), (dict(x=0), NULL), (dict(pre=0), NULL),
    (dict(dx=0, dw=0, db=0), NULL), (dict(d=MIS), ALIGN), (dict(w=MIS), ALIGN), (dict(x=MIS), ALIGN),
    (dict(pre=MIS), ALIGN), (dict(pre=MIS, act=0), ALIGN), (dict(dx=MIS), ALIGN), (dict(dw=MIS), ALIGN),
    (dict(db=MIS), ALIGN), (dict(ws=MIS), ALIGN), (dict(dxt=2), DTYPE), (dict(dwt=2), DTYPE), (dict(dbt=2), DTYPE),
    (dict(act=9), DTYPE), (dict(K=32), SHAPE), (dict(N=100), SHAPE), (dict(G=0), SHAPE), (dict(M=-5), SHAPE),
    (dict(G=4096, K=1 << 24, N=1 << 24), SHAPE), (dict(M=1 << 30, N=1 << 13), SHAPE),      # grids
    (dict(ws=0), WORKSPACE), (dict(wsb=256 + 100 * 192 * 2 + 4 * 9 * 192 - 1), WORKSPACE),
])
def test_linear_bwd_refusals(lib, kw, status):
    assert linear_bwd(lib, **kw) == status


def test_workspaces_of_the_product(lib):
    w = lib.gmm_workspace_bytes
    assert w(gmm.OP_BF16_LINEAR, 1000, 256, 128, 4) == 256
    # dpre, and partial sums of up to ceil(M / 32) + G + 1 items (128 rows an item from 2^25 values on)
    assert w(gmm.OP_BF16_LINEAR_BWD, 100, 128, 192, 4) == 256 + 100 * 192 * 2 + 4 * 9 * 192
    assert w(gmm.OP_BF16_LINEAR_BWD, 1 << 16, 512, 2048, 256) == 256 + (1 << 28) + 4 * (512 + 256 + 1) * 2048
    assert w(gmm.OP_BF16_LINEAR_BWD, 0, 128, 192, 4) == 256


def test_header_says_which_workspaces_hold_data(lib):
    read = lambda f: re.sub(r"[\s*]+", " ", open(os.path.join(ROOT, "include", f)).read())
    moe_h, gmm_h = read("gmm_moe.h"), read("gmm.h")
    rule = re.search(r"- Workspace:.*?- `stream`", gmm_h).group()
    for call, op in (("gmm_sort_tokens", gmm.OP_SORT_TOKENS), ("gmm_bf16_linear_bwd", gmm.OP_BF16_LINEAR_BWD)):
        assert lib.gmm_workspace_bytes(op, 100000, 256, 128, 4) > 256
        assert call in rule and "of its own until it has finished" in re.search(call + r" -- .*?GMM_API", moe_h).group()


# ------------------------------------------------------------- the binding --

class Lib:
    """Stands for the library: a call that gets this far would have launched."""

    def __getattr__(self, name):
        if name == "gmm_workspace_bytes":
            return lambda *args: 256

        def call(*args):
            raise AssertionError("%s was called" % name)
        return call


@pytest.fixture
def no_launch(monkeypatch):
    monkeypatch.setattr(moe, "load_library", Lib)


def t(shape, dt, dev="cpu"):
    return torch.zeros(shape, dtype=dt, device=dev)


T, E, k, K, M, G, N = 6, 32, 4, 64, 24, 8, 128
CALLS = {
    "gmm_route": dict(logits=(T, E, F32), k=k, bias=(E, F32), ids=(T, k, I32), weights=(T, k, F32)),
    "gmm_route_bwd": dict(dweights=(T, k, F32), logits=(T, E, BF), ids=(T, k, I32), out=(T, E, F32)),
    "gmm_sort_tokens": dict(ids=(T, k, I32), G=G, group_sizes=(G, I32), row_of=(T, k, I32), slot_of=(M, I32), ws=(4096, U8)),
    "gmm_dispatch": dict(x=(T, K, BF), row_of=(T, k, I32), slot_of=(M, I32), out=(M, K, BF)),
    "gmm_combine": dict(y=(M, K, BF), row_of=(T, k, I32), weights=(T, k, F32), residual=(T, K, F32), out=(T, K, F32)),
    "gmm_combine_bwd": dict(dout=(T, K, BF), y=(M, K, F32), row_of=(T, k, I32), slot_of=(M, I32), weights=(T, k, F32),
                            dy=(M, K, F32), dweights=(T, k, F32)),
    "gmm_bf16_linear": dict(lhs=(M, K, BF), rhs=(G, K, N, BF), group_sizes=(G, I32), bias=(G, N, F32), residual=(M, N, BF),
                            out=(M, N, BF), pre=(M, N, BF), ws=(256, U8)),
    "gmm_bf16_linear_bwd": dict(dout=(M, N, BF), rhs=(G, K, N, BF), group_sizes=(G, I32), lhs=(M, K, BF), pre=(M, N, BF),
                                dx=(M, K, F32), dw=(G, K, N, BF), db=(G, N, BF), ws=(1 << 16, U8)),
}
FIRST = dict(gmm_route="logits", gmm_route_bwd="logits", gmm_sort_tokens="ids", gmm_dispatch="x", gmm_combine="y",
             gmm_combine_bwd="dout", gmm_bf16_linear="lhs", gmm_bf16_linear_bwd="dout")


def args_of(call):
    return {n: t(v[:-1], v[-1]) if isinstance(v, tuple) else v for n, v in CALLS[call].items()}


TENSORS = [(c, n) for c in CALLS for n, v in CALLS[c].items() if isinstance(v, tuple)]


@pytest.mark.parametrize("call", CALLS)
def test_host_tensors_are_refused(no_launch, call):
    with pytest.raises(ValueError, match="not on a GPU"):
        getattr(gmm, call)(**args_of(call))


@pytest.mark.parametrize("call,name", TENSORS)
def test_another_device_is_refused(no_launch, call, name):
    a = args_of(call)
    a[name] = a[name].to("meta")
    with pytest.raises(ValueError, match="is on"):
        getattr(gmm, call)(**a)


@pytest.mark.parametrize("call,name", [(c, n) for c, n in TENSORS if n != "ws"])
def test_other_types_and_layouts_are_refused(no_launch, call, name):
    a = args_of(call)
    a[name] = a[name].double()
    with pytest.raises((TypeError, ValueError), match="dtype"):
        getattr(gmm, call)(**a)
    a = args_of(call)
    if a[name].dim() == 2:
        a[name] = a[name].t().contiguous().t()
        with pytest.raises(ValueError, match="contiguous"):
            getattr(gmm, call)(**a)


@pytest.mark.parametrize("call,name", [(c, n) for c, n in TENSORS if n not in ("ws", FIRST[c])])
def test_other_shapes_are_refused(no_launch, call, name):
    a = args_of(call)
    if call in ("gmm_dispatch", "gmm_combine_bwd") and name == "slot_of":
        a[name] = t((M + 1,), I32)
    else:
        a[name] = t((a[name].shape[0] + 1,) + tuple(a[name].shape[1:]), a[name].dtype)
    with pytest.raises(ValueError):
        getattr(gmm, call)(**a)


def test_the_tensors_device_is_the_current_one_of_a_call(monkeypatch):
    """A call on tensors of a device that is not the current one switches to it for the launch."""
    seen = []
    now = [0]

    class Switch:
        def __init__(self, dev):
            self.dev = dev

        def __enter__(self):
            self.before, now[0] = now[0], self.dev.index

        def __exit__(self, *exc):
            now[0] = self.before
    monkeypatch.setattr(moe, "_stream", lambda dev: 77)
    monkeypatch.setattr(moe, "_current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", Switch)
    fn = lambda *args: seen.append((now[0], args)) or 0
    moe._call(None, fn, torch.device("cuda", 0), 1, 2)
    moe._call(None, fn, torch.device("cuda", 1), 3)
    assert seen == [(0, (1, 2, 77)), (1, (3, 77))] and now == [0]


def test_names_are_checked(no_launch):
    with pytest.raises(ValueError, match="softplus"):
        gmm.gmm_route(t((T, E), F32), k, score="softplus")
    with pytest.raises(ValueError, match="swish"):
        gmm.gmm_bf16_linear(t((M, K), BF), t((G, K, N), BF), t((G,), I32), activation="swish")
    with pytest.raises(TypeError, match="float16"):
        gmm.gmm_bf16_linear(t((M, K), BF), t((G, K, N), BF), t((G,), I32), out_dtype=torch.float16)
    with pytest.raises(ValueError, match="tanh"):
        gmm.gmm_route_bwd(t((T, k), F32), t((T, E), F32), t((T, k), I32), score="tanh")
