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

from . import _DT, GmmError, load_library

OP_BF16_SWIGLU, OP_BF16_SWIGLU_BWD, OP_TGMM_MX8 = 16, 17, 18
FFN_EXPORTS = ("gmm_quantize_mx8", "gmm_dequantize_mx8", "gmm_bf16_swiglu", "gmm_bf16_swiglu_bwd", "tgmm_mx8")


_BYTES = (torch.uint8, torch.float8_e4m3fn)
_BF16 = (torch.bfloat16,)
_FLOAT = (torch.bfloat16, torch.float32)
_INT32 = (torch.int32,)
_U8 = (torch.uint8,)

_status_ws = {}    # device -> the status block of calls that were given no workspace
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


# A serving step's calls take a few microseconds on the device, so what the
# host does for each is kept small: addresses go to ctypes as integers, the
# stream comes from torch's raw lookup, and calls whose workspace is only the
# status word (nothing reads it when the caller gives no workspace) share one.

def _arg(t: Optional[torch.Tensor], want, dtypes: tuple, name: str, dev: torch.device) -> Optional[int]:
    """Address of t after checking its dtype, shape (want, unless None), layout and device: dev, that of the
    call's first operand, which _stream checks (a host address would fault in the kernel)."""
    if t is None:
        return None
    if t.dtype not in dtypes:
        raise TypeError("%s has dtype %s" % (name, t.dtype))
    if want is not None and t.shape != want:
        raise ValueError("%s is %s, not %s" % (name, tuple(t.shape), tuple(want)))
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    if t.device != dev:
        raise ValueError("%s is on %s, not on %s" % (name, t.device, dev))
    return t.data_ptr()


def _stream(dev: torch.device) -> int:
    """torch's current stream on dev."""
    if dev.type != "cuda":
        raise ValueError("the tensors are on %s, not on a GPU" % dev)
    if _raw_stream is not None and dev.index is not None:
        return _raw_stream(dev.index)
    return torch.cuda.current_stream(dev).cuda_stream


def _status(ws: Optional[torch.Tensor], dev: torch.device):
    """(address, bytes) of ws, or of the device's shared status block."""
    if ws is None:
        ws = _status_ws.get(dev)
        if ws is None:
            ws = _status_ws[dev] = torch.empty(256, dtype=torch.uint8, device=dev)
    elif not ws.is_contiguous():
        raise ValueError("tensors must be contiguous")
    elif ws.device != dev:
        raise ValueError("ws is on %s, not on %s" % (ws.device, dev))
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _check(lib, rc: int) -> None:
    if rc != 0:
        raise GmmError(rc, lib.gmm_last_error().decode())


def gmm_quantize_mx8(x: torch.Tensor, q: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None
                     ) -> Tuple[torch.Tensor, torch.Tensor]:
    """8-bit checkpoint of x [M,K] (bf16/fp32, K a multiple of 32): E4M3 codes
    uint8 [M,K] and E8M0 scales uint8 [M,K/32]."""
    lib = load_library()
    dev = x.device
    M, K = x.shape
    xp = _arg(x, None, _FLOAT, "x", dev)
    if q is None:
        q = torch.empty((M, K), dtype=torch.uint8, device=dev)
    if scale is None:
        scale = torch.empty((M, K // 32), dtype=torch.uint8, device=dev)
    _check(lib, lib.gmm_quantize_mx8(xp, _DT[x.dtype], M, K, _arg(q, (M, K), _BYTES, "q", dev),
                                     _arg(scale, (M, K // 32), _U8, "scale", dev), _stream(dev)))
    return q, scale


def gmm_dequantize_mx8(q: torch.Tensor, scale: torch.Tensor, out_dtype: torch.dtype = torch.bfloat16,
                       out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The values [M,K] (bf16 or fp32) of an 8-bit checkpoint."""
    lib = load_library()
    dev = q.device
    M, K = q.shape
    qp, sp = _arg(q, None, _BYTES, "q", dev), _arg(scale, (M, K // 32), _U8, "scale", dev)
    if out is None:
        out = torch.empty((M, K), dtype=out_dtype, device=dev)
    _check(lib, lib.gmm_dequantize_mx8(qp, sp, M, K, _arg(out, (M, K), _FLOAT, "out", dev), _DT[out.dtype],
                                       _stream(dev)))
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
    dev = lhs.device
    M, K = lhs.shape
    G, K2, N2 = rhs.shape
    if K2 != K or N2 % 2:
        raise ValueError("lhs K=%d but rhs %s" % (K, tuple(rhs.shape)))
    N = N2 // 2
    args = (_arg(lhs, None, _BF16, "lhs", dev), _arg(rhs, None, _BF16, "rhs", dev),
            _arg(group_sizes, (G,), _INT32, "group_sizes", dev), M, K, N, G)
    kept = (_arg(gu, (M, N2), _BF16, "gu", dev), _arg(gu_q, (M, N2), _BYTES, "gu_q", dev),
            _arg(gu_scale, (M, N2 // 32), _U8, "gu_scale", dev))
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=dev)
    _check(lib, lib.gmm_bf16_swiglu(*args, _arg(out, (M, N), _FLOAT, "out", dev), _DT[out.dtype], *kept,
                                    *_status(ws, dev), _stream(dev)))
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
    output recomputed from the kept P.  ws, if given (workspace(OP_BF16_SWIGLU_BWD,
    ...)), holds dP until the call's kernels have finished: a call that may run at
    the same time on another stream needs another one."""
    lib = load_library()
    dev = dh.device
    M, N = dh.shape
    G, K, N2 = rhs.shape
    if N2 != 2 * N:
        raise ValueError("dh N=%d but rhs %s" % (N, tuple(rhs.shape)))
    args = (_arg(dh, None, _BF16, "dh", dev), _arg(rhs, None, _BF16, "rhs", dev),
            _arg(group_sizes, (G,), _INT32, "group_sizes", dev), _arg(lhs, (M, K), _BF16, "lhs", dev),
            _arg(lhs_q, (M, K), _BYTES, "lhs_q", dev), _arg(lhs_scale, (M, K // 32), _U8, "lhs_scale", dev),
            _arg(gu, (M, N2), _BF16, "gu", dev), _arg(gu_q, (M, N2), _BYTES, "gu_q", dev),
            _arg(gu_scale, (M, N2 // 32), _U8, "gu_scale", dev), M, K, N, G)
    if dx is None and want_dx:
        dx = torch.empty((M, K), dtype=dx_dtype, device=dev)
    if dw is None and want_dw:
        dw = torch.empty((G, K, N2), dtype=dw_dtype, device=dev)
    if ws is None:
        ws = torch.empty(256 + 4 * M * N, dtype=torch.uint8, device=dev)
    _check(lib, lib.gmm_bf16_swiglu_bwd(
        *args, _arg(dx, (M, K), _FLOAT, "dx", dev), 0 if dx is None else _DT[dx.dtype],
        _arg(dw, (G, K, N2), _FLOAT, "dw", dev), 0 if dw is None else _DT[dw.dtype], _arg(h, (M, N), _BF16, "h", dev),
        *_status(ws, dev), _stream(dev)))
    return dx, dw


def tgmm_mx8(x_q: torch.Tensor, x_scale: torch.Tensor, dy: torch.Tensor, group_sizes: torch.Tensor,
             out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
             ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dW [G,K,N]: dW[g] = X_g^T dY_g with X kept as an 8-bit checkpoint
    (x_q [M,K], x_scale [M,K/32]) and dy [M,N] bf16."""
    lib = load_library()
    dev = x_q.device
    M, K = x_q.shape
    M2, N = dy.shape
    if M2 != M:
        raise ValueError("x has %d rows but dy has %d" % (M, M2))
    G = group_sizes.numel()
    args = (_arg(x_q, None, _BYTES, "x_q", dev), _arg(x_scale, (M, K // 32), _U8, "x_scale", dev),
            _arg(dy, None, _BF16, "dy", dev), _arg(group_sizes, (G,), _INT32, "group_sizes", dev), M, K, N, G)
    if out is None:
        out = torch.empty((G, K, N), dtype=out_dtype, device=dev)
    _check(lib, lib.tgmm_mx8(*args, _arg(out, (G, K, N), _FLOAT, "out", dev), _DT[out.dtype], *_status(ws, dev),
                             _stream(dev)))
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
