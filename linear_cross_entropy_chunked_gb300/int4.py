"""Linear layers with 4-bit weights and a scale per row and group, for answering
(lce_int4_quantize, lce_int4_linear). Argument marshalling only."""
from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple

import torch

from . import _binding as _b
from .fp8 import _check_dense_rows, _empty_out

GROUPS = (32, 64, 128)
_HALVES = (torch.bfloat16, torch.float16)


class Int4Weight(NamedTuple):
    """A linear layer's weight [V, D]: value k of a row is (q - 8) * scale[k // group], with q the low half
    of byte k / 2 for an even k, the high half for an odd one."""
    q: torch.Tensor       # [V, ceil(D / 2)] uint8, row stride a multiple of 16, at least ceil(D / 32) * 16
    scale: torch.Tensor   # [V, ceil(D / group)] bf16 or fp16
    group: int            # 32, 64 or 128


def _row_bytes(D):
    return -(-D // 32) * 16


def int4_weight(W, group: int = 128, scale_dtype=None, stream=None) -> Int4Weight:
    """W [V, D] (bf16, fp16 or fp32, unit column stride, any row stride) in 4 bits: a group's scale is a
    seventh of its largest magnitude, in scale_dtype (bf16 or fp16; default: W's, bf16 for fp32), within that type's
    smallest and largest positive number; the values are the nearest whole numbers within -8 .. 7, ties to even."""
    ldw = _check_dense_rows("W", W, _b._CE_DTYPES, "bfloat16, float16 or float32")
    if group not in GROUPS:
        raise ValueError(f"group must be one of {GROUPS}")
    if scale_dtype is None:
        scale_dtype = W.dtype if W.dtype in _HALVES else torch.bfloat16
    if scale_dtype not in _HALVES:
        raise TypeError("scale_dtype must be bfloat16 or float16")
    V, D = W.shape
    with _b._on(W.device, stream) as s:
        q = torch.empty((V, _row_bytes(D)), dtype=torch.uint8, device=W.device)
        scale = torch.empty((V, -(-D // group)), dtype=scale_dtype, device=W.device)
        _b._check(_b.lib().lce_int4_quantize(W.data_ptr(), _b._CE_DTYPES[W.dtype], ldw, V, D, group, q.data_ptr(),
                                             _row_bytes(D), scale.data_ptr(), _b._CE_DTYPES[scale_dtype],
                                             scale.shape[1], s), "lce_int4_quantize")
    return Int4Weight(q[:, :(D + 1) // 2], scale, group)


@functools.lru_cache(maxsize=1024)
def int4_workspace_size(M, D, group):
    """Bytes of a workspace for int4_linear of M tokens of D values (0: none is needed)."""
    out = ctypes.c_size_t(0)
    _b._check(_b.lib().lce_int4_linear_workspace_size(M, D, group, ctypes.byref(out)),
              "lce_int4_linear_workspace_size")
    return out.value


def _check_weight(w, X):
    """(V, row stride of q in bytes, row stride of the scales)."""
    D = X.shape[1]
    q, scale = w.q, w.scale
    if w.group not in GROUPS:
        raise ValueError(f"the weight's group must be one of {GROUPS}")
    if q.dtype != torch.uint8 or scale.dtype != X.dtype:
        raise TypeError("the weight's q must be uint8 and its scale of X's dtype")
    if q.device != X.device or scale.device != X.device:
        raise ValueError("X and the weight must be on one device")
    if q.dim() != 2 or q.shape[0] == 0 or q.shape[1] != (D + 1) // 2 or (q.shape[1] > 1 and q.stride(1) != 1):
        raise ValueError(f"the weight's q must be [V, {(D + 1) // 2}] for X's {D} columns")
    V = q.shape[0]
    if scale.shape != (V, -(-D // w.group)) or (scale.shape[1] > 1 and scale.stride(1) != 1):
        raise ValueError(f"the weight's scale must be [{V}, {-(-D // w.group)}]")
    ldq = q.stride(0) if V > 1 else max(_row_bytes(D), -(-q.stride(0) // 16) * 16)
    lds = scale.stride(0) if V > 1 else scale.shape[1]
    if ldq % 16 or ldq < _row_bytes(D) or q.data_ptr() % 16:
        raise ValueError("the weight's rows must lie on 16 bytes, with a stride of whole 32 values")
    if lds < scale.shape[1]:
        raise ValueError("the rows of the weight's scale must not overlap")
    if q.untyped_storage().nbytes() - q.storage_offset() < (V - 1) * ldq + _row_bytes(D):
        raise ValueError("the weight's last row must be padded to 16 bytes as the others are")
    return V, ldq, lds


def int4_linear(X, w: Int4Weight, out=None, ws=None, stream=None):
    """X W^T for the hidden states X [M, D] (bf16 or fp16, unit column stride, any row stride) and a weight in 4
    bits with scales of X's dtype: logits [M, V] in X's dtype, sums in fp32, rounded once. Fastest for few
    tokens, where it reads a quarter of a 16-bit weight's bytes. The logits' row stride is V rounded up to 16 bytes.
    out: where to write them (unit column stride). ws: a uint8 tensor of int4_workspace_size(M, D, w.group) bytes,
    whose device status read_status returns (where that is not 0); calls that may run at the same time need one each. No gradients: X may not
    require one."""
    ldx = _check_dense_rows("X", X, _HALVES, "bfloat16 or float16")
    if not isinstance(w, Int4Weight):
        raise TypeError("w must be an Int4Weight (int4_weight)")
    if X.requires_grad and torch.is_grad_enabled():
        raise ValueError("int4_linear has no gradients: detach X, or call it under torch.no_grad()")
    M, D = X.shape
    V, ldq, lds = _check_weight(w, X)
    if out is not None:
        ldc = _check_dense_rows("out", out, (X.dtype,), "of X's dtype") if out.numel() else out.stride(0)
        if out.shape != (M, V) or out.device != X.device:
            raise ValueError("out must be [M, V] on X's device")
        if out.requires_grad and torch.is_grad_enabled():
            raise ValueError("out may not require a gradient")
    with _b._on(X.device, stream) as s:
        Z = _empty_out(M, V, X.dtype, X.device) if out is None else out
        nbytes = int4_workspace_size(M, D, w.group)
        if ws is not None:
            if ws.device != X.device or ws.dtype != torch.uint8 or not ws.is_contiguous() or ws.numel() < nbytes \
                    or ws.data_ptr() % 16:
                raise ValueError(f"ws must be a contiguous, 16-byte aligned uint8 tensor of at least {nbytes} bytes")
        elif nbytes:
            ws = torch.empty(nbytes, dtype=torch.uint8, device=X.device)
        if M:
            _b._check(_b.lib().lce_int4_linear(
                X.data_ptr(), _b._CE_DTYPES[X.dtype], ldx, w.q.data_ptr(), ldq, w.scale.data_ptr(), lds, w.group, M,
                V, D, Z.data_ptr(), Z.stride(0) if M > 1 else V, None if ws is None else ws.data_ptr(),
                0 if ws is None else ws.numel(), s), "lce_int4_linear")
    if out is not None:
        _b._wrote((out,))
    return Z
