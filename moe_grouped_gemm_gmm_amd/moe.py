"""What stands around the experts' products of a mixture-of-experts layer
(include/gmm_moe.h): the router, tokens sorted by expert and back, and grouped
products with bias, activation and residual.

Argument marshalling only, in the manner of the package's other calls: outputs
are allocated with torch unless given, every call goes to torch's current
stream of the tensors' device, the checks are the C ABI's.  A layer forward:

    ids, weights = gmm_route(logits, k)
    group_sizes, row_of, slot_of = gmm_sort_tokens(ids, G)
    rows = gmm_dispatch(x, row_of, slot_of)
    y = ...                                       # the experts' products
    out = gmm_combine(y, row_of, weights=weights, residual=x)

and backward:

    dy, dweights = gmm_combine_bwd(dout, y, row_of, slot_of, weights)
    drows = ...                                   # the products' gradients
    dx = gmm_combine(drows, row_of, residual=dout)
    dlogits = gmm_route_bwd(dweights, logits, ids)
"""
import ctypes
import functools
from typing import Optional, Tuple

import torch

from . import _DT, ffn, load_library
from .ffn import _BF16, _FLOAT, _INT32, _arg, _check, _stream

OP_SORT_TOKENS, OP_BF16_LINEAR, OP_BF16_LINEAR_BWD = 32, 33, 34
MOE_EXPORTS = ("gmm_route", "gmm_route_bwd", "gmm_sort_tokens", "gmm_dispatch", "gmm_combine", "gmm_combine_bwd",
               "gmm_bf16_linear", "gmm_bf16_linear_bwd")
SCORES = {"softmax": 0, "sigmoid": 1}
ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
MAX_TOPK = 64

_F32 = (torch.float32,)


# A serving step's calls take a few microseconds on the device: outputs made
# here are not checked, and sizes of workspaces are asked for once.

def _out(t: Optional[torch.Tensor], shape, dtype: torch.dtype, dtypes: tuple, name: str, dev: torch.device):
    """(t, its address), t allocated unless given."""
    if t is None:
        if dtype not in dtypes:
            raise TypeError("%s has dtype %s" % (name, dtype))
        t = _empty(*shape, dtype=dtype, device=dev)   # sizes one by one: parsed faster than a tuple (1.3 us, 1.6)
        return t, t.data_ptr()
    return t, _arg(t, shape, dtypes, name, dev)


_empty = torch.empty
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _call(lib, fn, dev: torch.device, *args) -> None:
    """fn(*args, torch's current stream of dev), with dev as the current device."""
    stream = _stream(dev)
    if dev.index is None or _current_device() == dev.index:
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, stream)
    if rc:
        _check(lib, rc)


@functools.lru_cache(maxsize=512)
def _ws_bytes(op: int, M: int, K: int, N: int, G: int) -> int:
    return int(load_library().gmm_workspace_bytes(op, M, K, N, G))


def _work(ws: Optional[torch.Tensor], dev: torch.device, op: int, M: int, K: int, N: int, G: int):
    """(ws, its address, its bytes), ws allocated unless given or only the status block."""
    if ws is None:
        need = _ws_bytes(op, M, K, N, G)
        if need > 256:
            ws = _empty(need, dtype=torch.uint8, device=dev)
            return ws, ws.data_ptr(), need
    return (ws,) + ffn._status(ws, dev)


def _named(value: str, table: dict, what: str) -> int:
    code = table.get(value)
    if code is None:
        raise ValueError("%s %r is not one of %s" % (what, value, ", ".join(sorted(table))))
    return code


def gmm_route(logits: torch.Tensor, k: int, bias: Optional[torch.Tensor] = None, score: str = "softmax",
              normalize: bool = True, scale: float = 1.0, ids: Optional[torch.Tensor] = None,
              weights: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The k experts of every token and their weights: (ids int32 [T,k], weights
    fp32 [T,k]) from logits [T,E] (bf16/fp32).  score: "softmax" or "sigmoid" of
    the logits.  bias [E] fp32: the choice is by score + bias, the weights are of
    the score.  normalize: a token's weights sum to scale.  A logit of -infinity
    or NaN switches the expert off; a choice that cannot be made is -1 with
    weight 0."""
    lib = load_library()
    dev = logits.device
    T, E = logits.shape
    lp, bp = _arg(logits, None, _FLOAT, "logits", dev), _arg(bias, (E,), _F32, "bias", dev)
    kind = _named(score, SCORES, "score")
    ids, ip = _out(ids, (T, k), torch.int32, _INT32, "ids", dev)
    weights, wp = _out(weights, (T, k), torch.float32, _F32, "weights", dev)
    _call(lib, lib.gmm_route, dev, lp, _DT[logits.dtype], bp, T, E, k, kind, int(normalize), scale, ip, wp)
    return ids, weights


def gmm_route_bwd(dweights: torch.Tensor, logits: torch.Tensor, ids: torch.Tensor, score: str = "softmax",
                  normalize: bool = True, scale: float = 1.0, out_dtype: Optional[torch.dtype] = None,
                  out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of gmm_route's weights with respect to the logits, [T,E] (of the
    logits' dtype unless given), ids held fixed.  score, normalize and scale as
    given to gmm_route."""
    lib = load_library()
    dev = logits.device
    T, E = logits.shape
    T2, k = ids.shape
    if T2 != T:
        raise ValueError("logits has %d rows but ids has %d" % (T, T2))
    args = (_arg(dweights, (T, k), _F32, "dweights", dev), _arg(logits, None, _FLOAT, "logits", dev),
            _DT[logits.dtype], _arg(ids, None, _INT32, "ids", dev), T, E, k, _named(score, SCORES, "score"),
            int(normalize), scale)
    out, op = _out(out, (T, E), out_dtype or logits.dtype, _FLOAT, "out", dev)
    _call(lib, lib.gmm_route_bwd, dev, *args, op, _DT[out.dtype])
    return out


def gmm_sort_tokens(ids: torch.Tensor, G: int, first: int = 0, rows: Optional[int] = None,
                    group_sizes: Optional[torch.Tensor] = None, row_of: Optional[torch.Tensor] = None,
                    slot_of: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None
                    ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """The order of the slots (token t's choice j is slot t k + j) by expert:
    (group_sizes int32 [G], row_of int32 [T,k], slot_of int32 [rows]) from ids
    int32 [T,k].  Experts first .. first + G - 1 are sorted; a slot with another
    id has row -1.  rows (default T k): the sorted buffer's; slots past it have
    row -1 and device_status(ws) tells."""
    lib = load_library()
    dev = ids.device
    T, k = ids.shape
    M = T * k if rows is None else rows
    ip = _arg(ids, None, _INT32, "ids", dev)
    group_sizes, gp = _out(group_sizes, (max(G, 0),), torch.int32, _INT32, "group_sizes", dev)
    row_of, rp = _out(row_of, (T, k), torch.int32, _INT32, "row_of", dev)
    slot_of, sp = _out(slot_of, (max(M, 0),), torch.int32, _INT32, "slot_of", dev)
    ws, wp, wb = _work(ws, dev, OP_SORT_TOKENS, T * k, 0, 0, G)
    _call(lib, lib.gmm_sort_tokens, dev, ip, T, k, first, G, M, gp, rp, sp, wp, wb)
    return group_sizes, row_of, slot_of


def gmm_dispatch(x: torch.Tensor, row_of: torch.Tensor, slot_of: torch.Tensor, out: Optional[torch.Tensor] = None
                 ) -> torch.Tensor:
    """Tokens x [T,K] (bf16/fp32) in the sorted order, [M,K]; rows without a slot
    are zeros."""
    lib = load_library()
    dev = x.device
    T, K = x.shape
    T2, k = row_of.shape
    if T2 != T:
        raise ValueError("x has %d rows but row_of has %d" % (T, T2))
    M = slot_of.numel()
    args = (_arg(x, None, _FLOAT, "x", dev), _DT[x.dtype], _arg(row_of, None, _INT32, "row_of", dev),
            _arg(slot_of, (M,), _INT32, "slot_of", dev), T, k, M, K)
    out, op = _out(out, (M, K), x.dtype, (x.dtype,), "out", dev)
    _call(lib, lib.gmm_dispatch, dev, *args, op)
    return out


def gmm_combine(y: torch.Tensor, row_of: torch.Tensor, weights: Optional[torch.Tensor] = None,
                residual: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Results y [M,K] back to their tokens, [T,K] (of y's dtype unless given):
    residual + the sum of a token's rows, each times its weight (fp32 [T,k]).
    Without weights the gradient of gmm_dispatch."""
    lib = load_library()
    dev = y.device
    M, K = y.shape
    T, k = row_of.shape
    args = (_arg(y, None, _FLOAT, "y", dev), _DT[y.dtype], _arg(row_of, None, _INT32, "row_of", dev),
            _arg(weights, (T, k), _F32, "weights", dev))
    out, op = _out(out, (T, K), out_dtype or y.dtype, _FLOAT, "out", dev)
    _call(lib, lib.gmm_combine, dev, *args, _arg(residual, (T, K), (out.dtype,), "residual", dev), T, k, M, K, op,
          _DT[out.dtype])
    return out


def gmm_combine_bwd(dout: torch.Tensor, y: Optional[torch.Tensor], row_of: torch.Tensor, slot_of: torch.Tensor,
                    weights: Optional[torch.Tensor], want_dy: bool = True, want_dweights: bool = True,
                    dy_dtype: Optional[torch.dtype] = None, dy: Optional[torch.Tensor] = None,
                    dweights: Optional[torch.Tensor] = None
                    ) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    """Gradients of gmm_combine from dout [T,K]: (dy [M,K], dweights fp32 [T,k]).
    y is needed for dweights, weights for dy; dy has y's dtype (without y:
    dy_dtype, or dout's).  want_dy / want_dweights False leaves that one out
    (None).  The residual's gradient is dout."""
    lib = load_library()
    dev = dout.device
    T, K = dout.shape
    T2, k = row_of.shape
    if T2 != T:
        raise ValueError("dout has %d rows but row_of has %d" % (T, T2))
    M = slot_of.numel()
    dt = y.dtype if y is not None else (dy.dtype if dy is not None else dy_dtype or dout.dtype)
    args = (_arg(dout, None, _FLOAT, "dout", dev), _DT[dout.dtype], _arg(y, (M, K), _FLOAT, "y", dev), _DT.get(dt, -1),
            _arg(row_of, None, _INT32, "row_of", dev), _arg(slot_of, (M,), _INT32, "slot_of", dev),
            _arg(weights, (T, k), _F32, "weights", dev), T, k, M, K)
    yp = wp = None
    if dy is not None or want_dy:
        dy, yp = _out(dy, (M, K), dt, (dt,), "dy", dev)
    if dweights is not None or want_dweights:
        dweights, wp = _out(dweights, (T, k), torch.float32, _F32, "dweights", dev)
    _call(lib, lib.gmm_combine_bwd, dev, *args, yp, wp)
    return dy, dweights


def gmm_bf16_linear(lhs: torch.Tensor, rhs: torch.Tensor, group_sizes: torch.Tensor,
                    bias: Optional[torch.Tensor] = None, activation: str = "none",
                    residual: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
                    out: Optional[torch.Tensor] = None, pre: Optional[torch.Tensor] = None,
                    ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Grouped product with its epilogue: with pre = lhs [M,K] . rhs[g] [K,N] +
    bias[g] per group, activation(pre) + residual, [M,N].  bias [G,N] bf16 or
    fp32; activation "none", "relu", "silu", "gelu" or "gelu_tanh"; residual
    [M,N] of the output's type (it may be out itself).  pre [M,N] bf16, if given,
    receives pre for the backward pass."""
    lib = load_library()
    dev = lhs.device
    M, K = lhs.shape
    G, K2, N = rhs.shape
    if K2 != K:
        raise ValueError("lhs K=%d but rhs K=%d" % (K, K2))
    act = _named(activation, ACTIVATIONS, "activation")
    args = (_arg(lhs, None, _BF16, "lhs", dev), _arg(rhs, None, _BF16, "rhs", dev),
            _arg(group_sizes, (G,), _INT32, "group_sizes", dev), M, K, N, G, _arg(bias, (G, N), _FLOAT, "bias", dev),
            0 if bias is None else _DT[bias.dtype], act)
    pp = _arg(pre, (M, N), _BF16, "pre", dev)
    out, op = _out(out, (M, N), out_dtype, _FLOAT, "out", dev)
    _call(lib, lib.gmm_bf16_linear, dev, *args, _arg(residual, (M, N), (out.dtype,), "residual", dev), op,
          _DT[out.dtype], pp, *ffn._status(ws, dev))
    return out


def gmm_bf16_linear_bwd(dout: torch.Tensor, rhs: torch.Tensor, group_sizes: torch.Tensor,
                        lhs: Optional[torch.Tensor] = None, pre: Optional[torch.Tensor] = None,
                        activation: str = "none", dx_dtype: torch.dtype = torch.bfloat16,
                        dw_dtype: torch.dtype = torch.bfloat16, db_dtype: torch.dtype = torch.float32,
                        dx: Optional[torch.Tensor] = None, dw: Optional[torch.Tensor] = None,
                        db: Optional[torch.Tensor] = None, want_dx: bool = True, want_dw: bool = True,
                        want_db: bool = True, ws: Optional[torch.Tensor] = None
                        ) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor], Optional[torch.Tensor]]:
    """Backward of gmm_bf16_linear: (dx [M,K], dw [G,K,N], db [G,N]) from dout
    [M,N] bf16, the layer's input lhs (for dw) and, unless activation is "none",
    the kept pre.  want_dx / want_dw / want_db False leaves that gradient out
    (None).  The residual's gradient is dout.  ws, if given
    (workspace(OP_BF16_LINEAR_BWD, ...)), is used until the call's kernels have
    finished: a call that may run at the same time on another stream needs
    another one."""
    lib = load_library()
    dev = dout.device
    M, N = dout.shape
    G, K, N2 = rhs.shape
    if N2 != N:
        raise ValueError("dout N=%d but rhs N=%d" % (N, N2))
    args = (_arg(dout, None, _BF16, "dout", dev), _arg(rhs, None, _BF16, "rhs", dev),
            _arg(group_sizes, (G,), _INT32, "group_sizes", dev), _arg(lhs, (M, K), _BF16, "lhs", dev),
            _arg(pre, (M, N), _BF16, "pre", dev), _named(activation, ACTIVATIONS, "activation"), M, K, N, G)
    xp = wp = bp = None
    if dx is not None or want_dx:
        dx, xp = _out(dx, (M, K), dx_dtype, _FLOAT, "dx", dev)
    if dw is not None or want_dw:
        dw, wp = _out(dw, (G, K, N), dw_dtype, _FLOAT, "dw", dev)
    if db is not None or want_db:
        db, bp = _out(db, (G, N), db_dtype, _FLOAT, "db", dev)
    ws, sp, sb = _work(ws, dev, OP_BF16_LINEAR_BWD, M, K, N, G)
    _call(lib, lib.gmm_bf16_linear_bwd, dev, *args, xp, 0 if dx is None else _DT[dx.dtype], wp,
          0 if dw is None else _DT[dw.dtype], bp, 0 if db is None else _DT[db.dtype], sp, sb)
    return dx, dw, db


def _declare(lib) -> None:
    """ctypes signatures of this header's calls."""
    P, I, I64, SZ, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    lib.gmm_route.argtypes = [P, I, P, I64, I64, I64, I, I, F, P, P, P]
    lib.gmm_route_bwd.argtypes = [P, P, I, P, I64, I64, I64, I, I, F, P, I, P]
    lib.gmm_sort_tokens.argtypes = [P, I64, I64, I64, I64, I64, P, P, P, P, SZ, P]
    lib.gmm_dispatch.argtypes = [P, I, P, P, I64, I64, I64, I64, P, P]
    lib.gmm_combine.argtypes = [P, I, P, P, P, I64, I64, I64, I64, P, I, P]
    lib.gmm_combine_bwd.argtypes = [P, I, P, I, P, P, P, I64, I64, I64, I64, P, P, P]
    lib.gmm_bf16_linear.argtypes = [P, P, P, I64, I64, I64, I64, P, I, I, P, P, I, P, P, SZ, P]
    lib.gmm_bf16_linear_bwd.argtypes = [P, P, P, P, P, I, I64, I64, I64, I64, P, I, P, I, P, I, P, SZ, P]
    for name in MOE_EXPORTS:
        getattr(lib, name).restype = I
