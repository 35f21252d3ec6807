"""The gated expert block and 8-bit activation checkpoints (include/gmm_ffn.h).

Argument marshalling only, in the manner of the package's other calls:
outputs are allocated with torch unless given, every call goes to torch's
current stream, the checks are the C ABI's.  With a checkpoint of its input
and of its pre-activations a training step of one expert layer keeps 1.03
bytes per activation value:

    x_q, x_s = gmm_quantize_mx8(x)
    h = gmm_bf16_swiglu(x, w, gs, gu_q=gu_q, gu_scale=gu_s)
    ...
    dx, dw = gmm_bf16_swiglu_bwd(dh, w, gs, lhs_q=x_q, lhs_scale=x_s, gu_q=gu_q, gu_scale=gu_s)
"""
import ctypes
from typing import Optional, Tuple

import torch

from . import _check, _dt, _ptr, _stream, _ws, load_library

OP_BF16_SWIGLU, OP_BF16_SWIGLU_BWD, OP_TGMM_MX8 = 16, 17, 18
FFN_EXPORTS = ("gmm_quantize_mx8", "gmm_dequantize_mx8", "gmm_bf16_swiglu", "gmm_bf16_swiglu_bwd", "tgmm_mx8")


def _shape(t: Optional[torch.Tensor], want: tuple, name: str) -> None:
    if t is not None and tuple(t.shape) != want:
        raise ValueError("%s is %s, not %s" % (name, tuple(t.shape), want))


def _typed(t: Optional[torch.Tensor], dtypes: tuple, name: str) -> None:
    if t is not None and t.dtype not in dtypes:
        raise TypeError("%s has dtype %s" % (name, t.dtype))


_BYTES = (torch.uint8, torch.float8_e4m3fn)
_BF16 = (torch.bfloat16,)
_INT32 = (torch.int32,)
_U8 = (torch.uint8,)


def gmm_quantize_mx8(x: torch.Tensor, q: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None
                     ) -> Tuple[torch.Tensor, torch.Tensor]:
    """8-bit checkpoint of x [M,K] (bf16/fp32, K a multiple of 32): E4M3 codes
    uint8 [M,K] and E8M0 scales uint8 [M,K/32]."""
    lib = load_library()
    M, K = x.shape
    _typed(x, (torch.bfloat16, torch.float32), "x")
    _shape(q, (M, K), "q")
    _typed(q, _BYTES, "q")
    _shape(scale, (M, K // 32), "scale")
    _typed(scale, _U8, "scale")
    if q is None:
        q = torch.empty((M, K), dtype=torch.uint8, device=x.device)
    if scale is None:
        scale = torch.empty((M, K // 32), dtype=torch.uint8, device=x.device)
    _check(lib.gmm_quantize_mx8(_ptr(x), _dt(x), M, K, _ptr(q), _ptr(scale), _stream(x)))
    return q, scale


def gmm_dequantize_mx8(q: torch.Tensor, scale: torch.Tensor, out_dtype: torch.dtype = torch.bfloat16,
                       out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The values [M,K] (bf16 or fp32) of an 8-bit checkpoint."""
    lib = load_library()
    M, K = q.shape
    _typed(q, _BYTES, "q")
    _shape(scale, (M, K // 32), "scale")
    _typed(scale, _U8, "scale")
    _shape(out, (M, K), "out")
    if out is None:
        out = torch.empty((M, K), dtype=out_dtype, device=q.device)
    _check(lib.gmm_dequantize_mx8(_ptr(q), _ptr(scale), M, K, _ptr(out), _dt(out), _stream(q)))
    return out


def gmm_bf16_swiglu(lhs: torch.Tensor, rhs: torch.Tensor, group_sizes: torch.Tensor,
                    out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
                    gu: Optional[torch.Tensor] = None, gu_q: Optional[torch.Tensor] = None,
                    gu_scale: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gated expert block: with P = lhs [M,K] . rhs[g] [K,2N] (gate columns
    first) per group, silu(P[:, :N]) * P[:, N:], [M,N].  For the backward pass
    gu [M,2N] bf16, or gu_q [M,2N] uint8 and gu_scale [M,2N/32] uint8 (an 8-bit
    checkpoint), receives P."""
    lib = load_library()
    M, K = lhs.shape
    G, K2, N2 = rhs.shape
    if K2 != K or N2 % 2:
        raise ValueError("lhs K=%d but rhs %s" % (K, tuple(rhs.shape)))
    N = N2 // 2
    _typed(lhs, _BF16, "lhs")
    _typed(rhs, _BF16, "rhs")
    _shape(group_sizes, (G,), "group_sizes")
    _typed(group_sizes, _INT32, "group_sizes")
    _shape(out, (M, N), "out")
    _shape(gu, (M, N2), "gu")
    _typed(gu, _BF16, "gu")
    _shape(gu_q, (M, N2), "gu_q")
    _typed(gu_q, _BYTES, "gu_q")
    _shape(gu_scale, (M, N2 // 32), "gu_scale")
    _typed(gu_scale, _U8, "gu_scale")
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=lhs.device)
    ws, wsp, wsb = _ws(ws, OP_BF16_SWIGLU, M, K, N, G, lhs.device)
    _check(lib.gmm_bf16_swiglu(_ptr(lhs), _ptr(rhs), _ptr(group_sizes), M, K, N, G, _ptr(out), _dt(out),
                               _ptr(gu), _ptr(gu_q), _ptr(gu_scale), wsp, wsb, _stream(lhs)))
    return out


def gmm_bf16_swiglu_bwd(dh: torch.Tensor, rhs: torch.Tensor, group_sizes: torch.Tensor,
                        lhs: Optional[torch.Tensor] = None, lhs_q: Optional[torch.Tensor] = None,
                        lhs_scale: Optional[torch.Tensor] = None, gu: Optional[torch.Tensor] = None,
                        gu_q: Optional[torch.Tensor] = None, gu_scale: Optional[torch.Tensor] = None,
                        dx_dtype: torch.dtype = torch.bfloat16, dw_dtype: torch.dtype = torch.bfloat16,
                        dx: Optional[torch.Tensor] = None, dw: Optional[torch.Tensor] = None,
                        h: Optional[torch.Tensor] = None, want_dx: bool = True, want_dw: bool = True,
                        ws: Optional[torch.Tensor] = None
                        ) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    """Backward of gmm_bf16_swiglu: (dx [M,K], dw [G,K,2N]) from dh [M,N], the
    layer's input (lhs in bf16, or its checkpoint lhs_q, lhs_scale) and the
    kept P (gu in bf16, or gu_q, gu_scale).  want_dx / want_dw False leaves
    that gradient out (None).  h [M,N] bf16, if given, receives the forward's
    output recomputed from the kept P."""
    lib = load_library()
    M, N = dh.shape
    G, K, N2 = rhs.shape
    if N2 != 2 * N:
        raise ValueError("dh N=%d but rhs %s" % (N, tuple(rhs.shape)))
    for t, name in ((dh, "dh"), (rhs, "rhs"), (lhs, "lhs"), (gu, "gu"), (h, "h")):
        _typed(t, _BF16, name)
    for t, name in ((lhs_q, "lhs_q"), (gu_q, "gu_q")):
        _typed(t, _BYTES, name)
    for t, name in ((lhs_scale, "lhs_scale"), (gu_scale, "gu_scale")):
        _typed(t, _U8, name)
    _shape(group_sizes, (G,), "group_sizes")
    _typed(group_sizes, _INT32, "group_sizes")
    _shape(lhs, (M, K), "lhs")
    _shape(lhs_q, (M, K), "lhs_q")
    _shape(lhs_scale, (M, K // 32), "lhs_scale")
    _shape(gu, (M, N2), "gu")
    _shape(gu_q, (M, N2), "gu_q")
    _shape(gu_scale, (M, N2 // 32), "gu_scale")
    _shape(dx, (M, K), "dx")
    _shape(dw, (G, K, N2), "dw")
    _shape(h, (M, N), "h")
    if dx is None and want_dx:
        dx = torch.empty((M, K), dtype=dx_dtype, device=dh.device)
    if dw is None and want_dw:
        dw = torch.empty((G, K, N2), dtype=dw_dtype, device=dh.device)
    ws, wsp, wsb = _ws(ws, OP_BF16_SWIGLU_BWD, M, K, N, G, dh.device)
    _check(lib.gmm_bf16_swiglu_bwd(
        _ptr(dh), _ptr(rhs), _ptr(group_sizes), _ptr(lhs), _ptr(lhs_q), _ptr(lhs_scale), _ptr(gu), _ptr(gu_q),
        _ptr(gu_scale), M, K, N, G, _ptr(dx), 0 if dx is None else _dt(dx), _ptr(dw), 0 if dw is None else _dt(dw),
        _ptr(h), wsp, wsb, _stream(dh)))
    return dx, dw


def tgmm_mx8(x_q: torch.Tensor, x_scale: torch.Tensor, dy: torch.Tensor, group_sizes: torch.Tensor,
             out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
             ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dW [G,K,N]: dW[g] = X_g^T dY_g with X kept as an 8-bit checkpoint
    (x_q [M,K], x_scale [M,K/32]) and dy [M,N] bf16."""
    lib = load_library()
    M, K = x_q.shape
    M2, N = dy.shape
    if M2 != M:
        raise ValueError("x has %d rows but dy has %d" % (M, M2))
    G = group_sizes.numel()
    _typed(x_q, _BYTES, "x_q")
    _typed(x_scale, _U8, "x_scale")
    _typed(dy, _BF16, "dy")
    _typed(group_sizes, _INT32, "group_sizes")
    _shape(x_scale, (M, K // 32), "x_scale")
    _shape(out, (G, K, N), "out")
    if out is None:
        out = torch.empty((G, K, N), dtype=out_dtype, device=dy.device)
    ws, wsp, wsb = _ws(ws, OP_TGMM_MX8, M, K, N, G, dy.device)
    _check(lib.tgmm_mx8(_ptr(x_q), _ptr(x_scale), _ptr(dy), _ptr(group_sizes), M, K, N, G, _ptr(out), _dt(out),
                        wsp, wsb, _stream(dy)))
    return out


def _declare(lib) -> None:
    """ctypes signatures of this header's calls."""
    P, I, I64, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    lib.gmm_quantize_mx8.argtypes = [P, I, I64, I64, P, P, P]
    lib.gmm_dequantize_mx8.argtypes = [P, P, I64, I64, P, I, P]
    lib.gmm_bf16_swiglu.argtypes = [P, P, P, I64, I64, I64, I64, P, I, P, P, P, P, SZ, P]
    lib.gmm_bf16_swiglu_bwd.argtypes = [P] * 9 + [I64] * 4 + [P, I, P, I, P, P, SZ, P]
    lib.tgmm_mx8.argtypes = [P, P, P, P, I64, I64, I64, I64, P, I, P, SZ, P]
    for name in FFN_EXPORTS:
        getattr(lib, name).restype = I
