"""Sizes past what one launch can hold: HIP takes fewer than 2^32 threads a
dimension.  A call whose launches would not fit is refused with the other
shape errors, before anything is enqueued; the checkpoint calls split instead
(tested on the GPU)."""
import ctypes
import os
import re

import pytest

import moe_grouped_gemm_gmm_amd as gmm

SHAPE, WORKSPACE = 2, 5
A = 0x10000      # never dereferenced: the checks fail first
BIG = 1 << 45


def P(x):
    return ctypes.c_void_p(x) if x else None


@pytest.fixture(scope="module")
def lib():
    return gmm.load_library()


def bwd(lib, M, K, N, G, **kw):
    p = dict(dx=A, dw=A, ws=A)
    p.update(kw)
    return lib.gmm_bf16_swiglu_bwd(P(A), P(A), P(A), P(A), None, None, P(A), None, None, M, K, N, G, P(p["dx"]),
                                   1, P(p["dw"]), 1, None, P(p["ws"]), BIG, None)


def test_gradient_of_the_activation(lib):
    """One thread per 8 columns of a row: M N / 8 of them."""
    assert bwd(lib, 1 << 22, 64, 1 << 13, 4) == SHAPE                       # 2^32 threads
    assert bwd(lib, 1 << 22, 64, 1 << 13, 4, dx=0) == SHAPE
    # one row fewer fits (and is stopped by the next check, the workspace's)
    assert bwd(lib, (1 << 22) - 1, 64, 1 << 13, 4, ws=0) == WORKSPACE


def test_products(lib):
    """256 threads a tile of 128 x 128 of dX or dw, 128 x 64 of h."""
    assert bwd(lib, 1 << 22, 1 << 16, 64, 4) == SHAPE                       # dX: 2^24 tiles
    assert bwd(lib, 64, 1 << 18, 1 << 13, 64, dx=0) == SHAPE                # dw: 2^24 tiles
    assert lib.gmm_bf16_swiglu(P(A), P(A), P(A), 1 << 26, 64, 1 << 11, 4, P(A), 1, None, None, None, P(A), 256,
                               None) == SHAPE                               # h: 2^24 tiles
    assert lib.tgmm_mx8(P(A), P(A), P(A), P(A), 64, 1 << 18, 1 << 14, 64, P(A), 1, P(A), 256, None) == SHAPE


def test_headers_say_which_workspaces_hold_data(lib):
    """Calls that run at the same time may share a workspace only where it is the status block alone: each
    operation whose workspace is larger is named in gmm.h beside that permission, and in its own header."""
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    read = lambda f: re.sub(r"[\s*]+", " ", open(os.path.join(include, f)).read())
    gmm_h, ffn_h = read("gmm.h"), read("gmm_ffn.h")
    ops = dict(re.findall(r"GMM_OP_\w+ = (\d+),? / (\w+) /", gmm_h + ffn_h))
    assert len(ops) == 11
    rule = re.search(r"- Workspace:.*?- `stream`", gmm_h).group()
    size = re.search(r"gmm_workspace_bytes -- .*?GMM_API", gmm_h).group()
    data = [call for op, call in ops.items() if lib.gmm_workspace_bytes(int(op), 1000, 256, 128, 4) > 256]
    assert data == ["gmm_bf16_swiglu_bwd"]
    for call in data:
        assert call in rule and call in size
    assert "for every op" not in size
    own = re.search(r"gmm_bf16_swiglu_bwd -- .*?GMM_API", ffn_h).group()
    assert "workspace of its own" in own and "workspace of its own" in rule
