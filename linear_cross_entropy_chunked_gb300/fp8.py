"""Linear layers in 8-bit floating point (e4m3, one fp32 scale per block of 128 values along
the contraction): lce_fp8_quantize and lce_fp8_matmul. Argument marshalling only.

An operand is a pair (q, scale): q [R, C] float8_e4m3fn with a row stride that is a
multiple of 16, scale fp32 [R, ceil(C / 128)] (row blocks: activations, gradients) or
[ceil(R / 128), ceil(C / 128)] (tiles: weights), with any strides (row blocks come from
quantize_fp8 stored block by block: the product reads those of consecutive rows at once)."""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch
from torch.autograd.function import once_differentiable

from . import _binding as _b

BLOCK = 128
_WS_BYTES = 1024


class FP8Weight(NamedTuple):
    """A linear layer's weight [V, D] in tiles of 128 x 128, and (for the gradient of the
    layer's input) its transpose in the same form."""
    q: torch.Tensor                          # [V, D] float8_e4m3fn
    scale: torch.Tensor                      # [ceil(V / 128), ceil(D / 128)] fp32
    q_t: Optional[torch.Tensor] = None       # [D, V]
    scale_t: Optional[torch.Tensor] = None   # [ceil(D / 128), ceil(V / 128)]


def _blocks(n):
    return -(-n // BLOCK)


def _pad16(n):
    return -(-n // 16) * 16


def _check_dense_rows(name, t, dtypes, what):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {what}")
    if t.dim() != 2 or t.shape[1] == 0 or (t.stride(1) != 1 and t.shape[1] > 1):
        raise ValueError(f"{name} must be 2-D with unit column stride")
    ld = t.stride(0) if t.shape[0] > 1 else t.shape[1]
    if ld < t.shape[1]:
        raise ValueError(f"the rows of {name} must not overlap")
    return ld


def _operand(R, C, tiles, dev):
    """(q [R, C] with padded rows, scale) for an operand of that shape."""
    ld = _pad16(C)
    q = torch.empty((R, ld), dtype=torch.float8_e4m3fn, device=dev)
    if tiles:
        scale = torch.empty((_blocks(R), _blocks(C)), dtype=torch.float32, device=dev)
    else:   # stored block by block
        scale = torch.empty((_blocks(C), R), dtype=torch.float32, device=dev).t()
    return q if ld == C else q[:, :C], scale


def _quantize(X, tiles, own, transposed, s):
    """((q, scale) or None, the same of X^T or None) on the current device and stream."""
    R, C = X.shape
    ld = X.stride(0) if R > 1 else C
    q = scale = qt = scale_t = None
    if own:
        q, scale = _operand(R, C, tiles, X.device)
    if transposed:
        qt, scale_t = _operand(C, R, tiles, X.device)
    if R:
        _b._check(_b.lib().lce_fp8_quantize(
            X.data_ptr(), _b._CE_DTYPES[X.dtype], ld, R, C, tiles,
            q.data_ptr() if own else None, _pad16(C), scale.data_ptr() if own else None,
            qt.data_ptr() if transposed else None, _pad16(R), scale_t.data_ptr() if transposed else None,
            s), "lce_fp8_quantize")
    return (q, scale), (qt, scale_t)


def quantize_fp8(X, tiles: bool = False, transpose: bool = False, stream=None):
    """(q, scale) of X [R, C] (bf16, fp16 or fp32, unit column stride, any row stride), or
    of X^T with transpose=True, in row blocks of 128 values or (tiles=True) in tiles of
    128 x 128. The scale is the smallest power of two under which the block's largest
    finite value is at most 448, so only e4m3's rounding (to nearest, ties to even) loses
    anything; infinities and NaN become NaN."""
    _check_dense_rows("X", X, _b._CE_DTYPES, "bfloat16, float16 or float32")
    if transpose and X.shape[0] == 0:
        raise ValueError("X has no rows to contract over")
    with _b._on(X.device, stream) as s:
        own, t = _quantize(X, tiles, not transpose, transpose, s)
    return t if transpose else own


def fp8_weight(W, transpose: bool = True, stream=None) -> FP8Weight:
    """The weight W [V, D] (bf16, fp16 or fp32) in tiles; with transpose also its
    transpose, which the gradient of the layer's input needs."""
    _check_dense_rows("W", W, _b._CE_DTYPES, "bfloat16, float16 or float32")
    if W.shape[0] == 0:
        raise ValueError("W has no rows")
    with _b._on(W.device, stream) as s:
        own, t = _quantize(W, True, True, transpose, s)
    return FP8Weight(*own, *t)


def _check_operand(name, q, scale, rows_only):
    """Row stride, and whether the scales are per row."""
    ld = _check_dense_rows(name, q, (torch.float8_e4m3fn,), "float8_e4m3fn")
    if q.shape[0] > 1 and ld % 16:
        raise ValueError(f"{name}'s row stride must be a multiple of 16 (pad its rows)")
    if q.data_ptr() % 16:
        raise ValueError(f"{name} must start on a 16-byte boundary")
    R, KB = q.shape[0], _blocks(q.shape[1])
    if scale.dtype != torch.float32 or scale.device != q.device:
        raise ValueError(f"{name}'s scale must be a float32 tensor on its device")
    rows = scale.shape == (R, KB)
    if not rows and (rows_only or scale.shape != (_blocks(R), KB)):
        raise ValueError(f"{name}'s scale must be [{R}, {KB}] (rows)" +
                         ("" if rows_only else f" or [{_blocks(R)}, {KB}] (tiles)") +
                         f", not {list(scale.shape)}")
    return _pad16(ld) if R <= 1 else ld, rows


def fp8_matmul_workspace_size(M, N, K, rows=False):
    """Bytes of a workspace for fp8_matmul ([M, K] by [N, K]; rows: b's scales are per row) with which
    products with few tiles and a long K are shared out along K, on the current device."""
    out = ctypes.c_size_t(0)
    _b._check(_b.lib().lce_fp8_matmul_best_workspace_size(M, N, K, 1 if rows else 0, ctypes.byref(out)),
              "lce_fp8_matmul_best_workspace_size")
    return out.value


def _matmul(a, a_scale, lda, b, b_scale, ldb, b_rows, out, ws, s):
    M, K = a.shape
    N = b.shape[0]
    ldc = out.stride(0) if M > 1 else -(-N // 8) * 8
    if ws is None:
        nbytes = fp8_matmul_workspace_size(M, N, K, b_rows) if M > BLOCK else _WS_BYTES
        ws = torch.empty(nbytes, dtype=torch.uint8, device=a.device)
    _b._check(_b.lib().lce_fp8_matmul(a.data_ptr(), lda, a_scale.data_ptr(), *a_scale.stride(), b.data_ptr(),
                                      ldb, b_scale.data_ptr(), *b_scale.stride(), 1 if b_rows else 0, M, N, K,
                                      out.data_ptr(), ldc, _b._CE_DTYPES[out.dtype], ws.data_ptr(), ws.numel(),
                                      s), "lce_fp8_matmul")
    return out


def _empty_out(M, N, dtype, dev):
    """[M, N]; the row stride is rounded up so that every row starts on 16 bytes."""
    per = 16 // dtype.itemsize
    return torch.empty_strided((M, N), (-(-N // per) * per, 1), dtype=dtype, device=dev)


def fp8_matmul(a, a_scale, b, b_scale, out_dtype=torch.bfloat16, out=None, ws=None, stream=None):
    """a @ b.T in e4m3: a [M, K] with scales per row and block of 128 [M, ceil(K / 128)],
    b [N, K] with scales per row and block or per tile [ceil(N / 128), ceil(K / 128)]; any
    fp32 scales, fp32 sums, rounded once to out_dtype (bf16, fp16 or fp32). The result's
    row stride is N rounded up to 16 bytes. out: where to write it (row stride a multiple of
    16 bytes). ws: a uint8 tensor of at least 1024 bytes whose device status read_status returns
    (fp8_matmul_workspace_size says with how many no product is slower than without ws); calls
    that may run at the same time need one each."""
    lda, _ = _check_operand("a", a, a_scale, True)
    ldb, b_rows = _check_operand("b", b, b_scale, False)
    if a.shape[1] != b.shape[1] or a.device != b.device:
        raise ValueError(f"a{tuple(a.shape)} and b{tuple(b.shape)} must share their columns and device")
    if out is not None:
        ldc = _check_dense_rows("out", out, _b._CE_DTYPES, "bfloat16, float16 or float32") \
            if out.numel() else out.stride(0)
        if out.shape != (a.shape[0], b.shape[0]) or out.device != a.device:
            raise ValueError("out must be [M, N] on the operands' device")
        if out.data_ptr() % 16 or (out.shape[0] > 1 and ldc * out.element_size() % 16):
            raise ValueError("out's rows must start on 16-byte boundaries")
    elif out_dtype not in _b._CE_DTYPES:
        raise TypeError("out_dtype must be bfloat16, float16 or float32")
    if ws is not None and (ws.device != a.device or ws.dtype != torch.uint8 or not ws.is_contiguous()
                           or ws.numel() < _WS_BYTES or ws.data_ptr() % 16):
        raise ValueError(f"ws must be a contiguous, 16-byte aligned uint8 tensor of at least {_WS_BYTES} bytes")
    with _b._on(a.device, stream) as s:
        if out is None:
            return _matmul(a, a_scale, lda, b, b_scale, ldb, b_rows,
                           _empty_out(a.shape[0], b.shape[0], out_dtype, a.device), ws, s)
        _matmul(a, a_scale, lda, b, b_scale, ldb, b_rows, out, ws, s)
    _b._wrote((out,))
    return out


def _collect(status, ws, at=0):
    """Adds the device status in the workspace header at byte `at` of ws to the caller's."""
    status[:4].view(torch.int32).bitwise_or_(ws[at:at + 4].view(torch.int32))


def _logits(X, q, scale, status, s):
    """X W^T on the current device and stream, for W's tiles."""
    M, D = X.shape
    V = q.shape[0]
    Z = _empty_out(M, V, X.dtype, X.device)
    code = _b._CE_DTYPES[X.dtype]
    nbytes = _WS_BYTES + (4 * M * _blocks(D) + 1023) // 1024 * 1024 + M * _pad16(D)
    parts = _ws_bytes(M, V, D) - _WS_BYTES   # (shared out along D as with a weight that is quantised here)
    if parts:
        nbytes = (nbytes + 1023) // 1024 * 1024 + parts
    ws = torch.empty(nbytes, dtype=torch.uint8, device=X.device)
    _b._check(_b.lib().lce_fp8_linear(
        X.data_ptr(), code, X.stride(0) if M > 1 else D, q.data_ptr(), q.stride(0) if V > 1 else _pad16(D),
        scale.data_ptr(), *scale.stride(), M, V, D, Z.data_ptr(), Z.stride(0) if M > 1 else -(-V // 8) * 8, code,
        ws.data_ptr(), nbytes, s), "lce_fp8_linear")
    if status is not None:
        _collect(status, ws)
    return Z


class _At(NamedTuple):
    """An operand in a buffer of several: addresses, row stride and the scales' strides."""
    q: int
    ld: int
    scale: int
    row: int
    block: int
    end: int


def _at(base, R, C, tiles):
    """Lays the operand [R, C] out from address `base` on (256-byte steps)."""
    ld = _pad16(C)
    scale = base + (R * ld + 255) // 256 * 256
    kb = _blocks(C)
    end = scale + (4 * (_blocks(R) if tiles else R) * kb + 255) // 256 * 256
    return _At(base, ld, scale, kb if tiles else 1, 1 if tiles else R, end)


def _quantize_at(X, tiles, own, transposed, s):
    R, C = X.shape
    if R:
        _b._check(_b.lib().lce_fp8_quantize(
            X.data_ptr(), _b._CE_DTYPES[X.dtype], X.stride(0) if R > 1 else C, R, C, tiles,
            own.q if own else None, _pad16(C), own.scale if own else None,
            transposed.q if transposed else None, _pad16(R), transposed.scale if transposed else None, s),
            "lce_fp8_quantize")


def _matmul_at(a, b, b_rows, M, N, K, out, ws, ws_bytes, s):
    ldc = out.stride(0) if M > 1 else -(-N // 8) * 8
    _b._check(_b.lib().lce_fp8_matmul(a.q, a.ld, a.scale, a.row, a.block, b.q, b.ld, b.scale, b.row, b.block,
                                      1 if b_rows else 0, M, N, K, out.data_ptr(), ldc,
                                      _b._CE_DTYPES[out.dtype], ws, ws_bytes, s), "lce_fp8_matmul")


def _ws_bytes(M, N, K):
    return fp8_matmul_workspace_size(M, N, K) if M > BLOCK else _WS_BYTES


class FP8LinearFunction(torch.autograd.Function):
    """Z = X W^T with X in row blocks and W in tiles of e4m3; rounding is passed through:
    dX = dZ W (dZ in row blocks, W^T in tiles) and, for a trained W, dW = dZ^T X (both in
    blocks along the rows of X). What lives as long is allocated at once: the operands of this
    pass in one buffer, those of the backward pass in another."""

    @staticmethod
    def forward(ctx, X, W, q, scale, q_t, scale_t, status=None):
        need_dX, need_dW = ctx.needs_input_grad[0], ctx.needs_input_grad[1]
        ctx.x_dtype, ctx.w_dtype, ctx.status = X.dtype, None if W is None else W.dtype, status
        with _b._on(X.device, None) as s:
            if W is None:
                ctx.save_for_backward(q_t, scale_t)
                return _logits(X, q, scale, status, s)
            (M, D), V = X.shape, W.shape[0]
            x, w = _at(0, M, D, False), _at(0, V, D, True)
            wt = _at(0, D, V, True).end if need_dX else 0
            xt = _at(0, D, M, False).end if need_dW else 0
            nbytes = _ws_bytes(M, V, D)
            here = torch.empty(x.end + w.end + nbytes, dtype=torch.uint8, device=X.device)
            kept = torch.empty(wt + xt, dtype=torch.uint8, device=X.device)
            x = _at(here.data_ptr(), M, D, False)
            w = _at(x.end, V, D, True)
            _quantize_at(W, True, w, _at(kept.data_ptr(), D, V, True) if need_dX else None, s)
            _quantize_at(X, False, x, _at(kept.data_ptr() + wt, D, M, False) if need_dW else None, s)
            Z = _empty_out(M, V, X.dtype, X.device)
            _matmul_at(x, w, False, M, V, D, Z, w.end, nbytes, s)
            if status is not None:
                _collect(status, here, w.end - here.data_ptr())
        ctx.save_for_backward(kept)
        ctx.D = D
        return Z

    @staticmethod
    @once_differentiable
    def backward(ctx, dZ):
        need_dX, need_dW = ctx.needs_input_grad[0], ctx.needs_input_grad[1]
        if not (need_dX or need_dW):
            return (None,) * 7
        if dZ.stride(1) != 1 or (dZ.shape[0] > 1 and dZ.stride(0) < dZ.shape[1]):
            dZ = dZ.contiguous()
        M, V = dZ.shape
        dX = dW = None
        with _b._on(dZ.device, None) as s:
            if ctx.w_dtype is None:
                wq, ws = ctx.saved_tensors
                D = wq.shape[0]
                wt = _At(wq.data_ptr(), wq.stride(0) if D > 1 else _pad16(V), ws.data_ptr(), *ws.stride(), 0)
            else:
                (kept,), D = ctx.saved_tensors, ctx.D
                wt = _at(kept.data_ptr(), D, V, True)
                xt = _at(wt.end if need_dX else kept.data_ptr(), D, M, False)
            nbytes = max(_ws_bytes(M, D, V) if need_dX else 0, _WS_BYTES)
            z, zt = (_at(0, M, V, False).end if need_dX else 0), (_at(0, V, M, False).end if need_dW else 0)
            here = torch.empty(z + zt + nbytes, dtype=torch.uint8, device=dZ.device)
            at = here.data_ptr()
            z, zt, at = _at(at, M, V, False), _at(at + z, V, M, False), at + z + zt
            _quantize_at(dZ, False, z if need_dX else None, zt if need_dW else None, s)
            if need_dX:
                dX = _empty_out(M, D, ctx.x_dtype, dZ.device)
                _matmul_at(z, wt, False, M, D, V, dX, at, nbytes, s)
                if ctx.status is not None:
                    _collect(ctx.status, here, at - here.data_ptr())
            if need_dW:
                if M == 0:
                    dW = torch.zeros(V, D, dtype=ctx.w_dtype, device=dZ.device)
                else:
                    dW = _empty_out(V, D, ctx.w_dtype, dZ.device)
                    _matmul_at(zt, xt, True, V, D, M, dW, at, nbytes, s)
                    if ctx.status is not None:
                        _collect(ctx.status, here, at - here.data_ptr())
        return dX, dW, None, None, None, None, None


def fp8_linear(X, W, status=None):
    """X W^T computed in e4m3 with blocks of 128, in X's dtype: logits [M, V] for the hidden
    states X [M, D] (bf16, fp16 or fp32). W: a weight [V, D] (bf16, fp16 or fp32), quantised in
    the call and differentiable, or an FP8Weight, which is frozen (its transpose is needed
    where X requires a gradient). Differentiable in X and W; the gradients are
    products in e4m3 too, and have no derivatives themselves. The logits' row stride is V rounded up
    to 16 bytes, the gradients' D. status: a uint8 tensor of at least 1024 bytes, zeros at first, that collects the device
    status of the layer's products, the forward's and the backward's, until read_status(status)
    returns and clears it (a product whose bounded wait ran out has wrong results; without `status`
    that is not noticed). (A backward pass
    is captured into a CUDA graph as any other of torch's: no eager graph of the same leaves may
    live meanwhile; X.detach().requires_grad_() gives a leaf of its own.)"""
    _check_dense_rows("X", X, _b._CE_DTYPES, "bfloat16, float16 or float32")
    if status is not None and (status.device != X.device or status.dtype != torch.uint8 or status.data_ptr() % 16
                               or not status.is_contiguous() or status.dim() != 1 or status.numel() < _WS_BYTES):
        raise ValueError(f"status must be a 16-byte aligned uint8 tensor of at least {_WS_BYTES} bytes on the device of X")
    D = X.shape[1]
    if isinstance(W, FP8Weight):
        q, scale = W.q, W.scale
        _check_operand("W", q, scale, False)
        V = q.shape[0]
        if q.shape[1] != D or q.device != X.device:
            raise ValueError(f"X{tuple(X.shape)} and W{tuple(q.shape)} must share their columns and device")
        if scale.shape != (_blocks(V), _blocks(D)):
            raise ValueError("the scales of W must be per tile of 128 x 128")
        if not (X.requires_grad and torch.is_grad_enabled()):
            with _b._on(X.device, None) as s:
                return _logits(X, q, scale, status, s)
        if W.q_t is None or W.scale_t is None:
            raise ValueError("the gradient of X needs W's transpose (fp8_weight(W, transpose=True))")
        _check_operand("W's transpose", W.q_t, W.scale_t, False)
        if W.q_t.shape != (D, V) or W.q_t.device != X.device or W.scale_t.shape != (_blocks(D), _blocks(V)):
            raise ValueError("W's transpose must be [D, V] in tiles of 128 x 128")
        return FP8LinearFunction.apply(X, None, q, scale, W.q_t, W.scale_t, status)
    _check_dense_rows("W", W, _b._CE_DTYPES, "bfloat16, float16 or float32, or an FP8Weight")
    if D != W.shape[1] or X.device != W.device or W.shape[0] == 0:
        raise ValueError(f"X{tuple(X.shape)} and W{tuple(W.shape)} must share their columns and device")
    if not torch.is_grad_enabled():   # (no transposes for a backward pass that cannot come)
        X, W = X.detach(), W.detach()
    return FP8LinearFunction.apply(X, W, None, None, None, None, status)
