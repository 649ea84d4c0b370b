"""The global norm of a list of gradients, and clipping by it (lce_grad_norm,
lce_clip_grad_norm). Argument marshalling only (and, for rows that are padded, dense copies)."""
from __future__ import annotations

import ctypes
import math
import operator
from array import array

import torch

from . import _binding as _b

_dtype = operator.attrgetter("dtype")
NORM_KINDS = {2.0: 0, math.inf: 1, 1.0: 2}


def _dense(t) -> bool:
    """Whether the tensor's values fill one range of memory, in whatever order."""
    if t.is_contiguous():
        return True
    want = 1
    for stride, size in sorted((st, n) for st, n in zip(t.stride(), t.shape) if n != 1):
        if stride != want:
            return False
        want *= size
    return True


def _padded(t) -> bool:
    """Whether the tensor has rows rounded up to 16 bytes, as fp8_linear's gradients and logits."""
    per = 16 // t.element_size()
    return t.dim() == 2 and t.stride(1) == 1 and t.stride(0) == -(-t.shape[1] // per) * per


def _tensors(grads, what):
    """(list of the tensors, device, whether all are contiguous (None: some have padded rows),
    and their addresses, sizes and dtype codes). Lists of hundreds are usual: one pass in C per property."""
    grads = [grads] if isinstance(grads, torch.Tensor) else list(grads)
    if not grads:
        raise ValueError(f"{what} is empty")
    T = torch.Tensor
    devices = set(map(T.get_device, grads))   # -1: not on a GPU
    if len(devices) > 1 or -1 in devices:
        if -1 in devices:
            raise ValueError(f"{what} must be CUDA tensors (there is no CPU path)")
        raise ValueError(f"{what} must be on one device")
    codes = _b._CE_DTYPES
    dtypes = set(map(_dtype, grads))
    if not dtypes <= codes.keys():
        raise TypeError(f"{what} must be bfloat16, float16 or float32")
    plain = all(map(T.is_contiguous, grads))
    if not plain:
        gaps = [g for g in grads if not _dense(g)]
        if not all(map(_padded, gaps)):
            raise ValueError(f"{what} must fill their memory (contiguous or permuted, no gaps but of rows that "
                             "are padded to 16 bytes)")
        if gaps:
            plain = None
    return (grads, grads[0].device, plain, array("Q", map(T.data_ptr, grads)), array("q", map(T.numel, grads)),
            array("i", [codes[dtypes.pop()]]) * len(grads) if len(dtypes) == 1
            else array("i", [codes[g.dtype] for g in grads]))


def _kind(norm_type):
    kind = NORM_KINDS.get(float(norm_type))
    if kind is None:
        raise ValueError("norm_type must be 1, 2 or inf")
    return kind


def _at(a):
    """Address of an array's items (which must outlive the call)."""
    return a.buffer_info()[0]


def _workspace(n, ws, dev):
    if ws is not None:
        if ws.device != dev or not ws.is_contiguous():
            raise ValueError("ws must be a contiguous tensor on the gradients' device")
        return ws, ws.numel() * ws.element_size()
    nbytes = ctypes.c_size_t(0)
    _b._check(_b.lib().lce_grad_norm_workspace_size(n, ctypes.byref(nbytes)), "lce_grad_norm_workspace_size")
    return torch.empty(nbytes.value, dtype=torch.uint8, device=dev), nbytes.value


def _copies(tensors, empty=False):
    """The tensors with dense copies in the place of those that have gaps."""
    return [t if _dense(t) else torch.empty(t.shape, dtype=t.dtype, device=t.device) if empty else t.contiguous()
            for t in tensors]


def _refuse_overlaps(grads, out):
    """As the library does for the ranges that it gets: a tensor that is written may lie over no
    other of the call, except that an output may be its own gradient. Rows count with their padding."""
    def span(t):
        end = sum((n - 1) * st for n, st in zip(t.shape, t.stride())) + 1
        return t.data_ptr(), t.data_ptr() + end * t.element_size()
    ranges = []
    for i, g in enumerate(grads):
        if g.numel():
            o = g if out is None else out[i]
            ranges.append((*span(o), True))
            if span(o) != span(g):
                ranges.append((*span(g), False))
    end = written_end = 0
    for a, b, written in sorted(ranges):
        if a < (end if written else written_end):
            raise _b.LCEError(1, "clip_grad_norm: tensors overlap")
        end = max(end, b)
        if written:
            written_end = max(written_end, b)


def _clip_copies(grads, out, max_norm, norm_type, eps, ws):
    """clip_grad_norm, on the current device and stream, where some rows are padded."""
    _refuse_overlaps(grads, out)
    src = _copies(grads)
    dst = None if out is None else _copies(out, empty=True)
    norm = clip_grad_norm(src, max_norm, norm_type, eps, dst, ws)
    with torch.no_grad():
        for t, c in zip(grads, src) if out is None else zip(out, dst):
            if c is not t:
                t.copy_(c)
    return norm


def grad_norm(grads, norm_type=2.0, ws=None, stream=None):
    """The norm (1, 2 or inf) over all values of the gradients, a tensor or a list of
    tensors (bf16, fp16 and fp32 may be mixed; contiguous or permuted; rows that are padded to
    16 bytes, as fp8_linear's gradients, are copied first): a device fp32 scalar."""
    kind = _kind(norm_type)
    grads, dev, plain, ptrs, sizes, codes = _tensors(grads, "grads")
    if plain is None:
        with _b._on(dev, stream):
            return grad_norm(_copies(grads), norm_type, ws)
    n = len(ptrs)
    with _b._on(dev, stream) as s:
        ws, ws_bytes = _workspace(n, ws, dev)
        norm = torch.empty((), dtype=torch.float32, device=dev)
        _b._check(_b.lib().lce_grad_norm(_at(ptrs), _at(sizes), _at(codes), n, kind, norm.data_ptr(), ws.data_ptr(),
                                         ws_bytes, s), "lce_grad_norm")
    return norm


def clip_grad_norm(grads, max_norm, norm_type=2.0, eps=1e-6, out=None, ws=None, stream=None):
    """Scales the gradients (a tensor or a list, bf16, fp16 and fp32 may be mixed) by
    min(1, max_norm / (norm + eps)), in place or into the tensors `out` of the same
    dtypes, sizes and layouts, and returns their norm (1, 2 or inf over all values; a device fp32
    scalar; the host does not wait). Rows that are padded to 16 bytes, as fp8_linear's gradients, go
    through dense copies. The factor is formed on the device: gradients
    whose norm is below max_norm stay as they are and are not written in place. A norm
    that is NaN (infinite) makes the factor NaN (0). To autograd the tensors count as written
    either way: a backward pass that saved one of them refuses to run afterwards."""
    kind = _kind(norm_type)
    max_norm, eps = float(max_norm), float(eps)
    if not max_norm >= 0.0 or not 0.0 <= eps < math.inf:
        raise ValueError("max_norm must not be negative, and eps finite and not negative")
    grads, dev, plain, ptrs, sizes, codes = _tensors(grads, "grads")
    n = len(ptrs)
    dst, padded = None, plain is None
    if out is not None:
        out, out_dev, out_plain, out_ptrs, out_sizes, out_codes = _tensors(out, "out")
        padded = padded or out_plain is None
        if out_dev != dev or out_sizes != sizes or out_codes != codes or not (padded or plain and out_plain or all(
                o.shape == g.shape and o.stride() == g.stride() for o, g in zip(out, grads))):
            raise ValueError("out must match the gradients in number, device, dtypes, sizes and layouts")
        dst = _at(out_ptrs)
    if padded:
        with _b._on(dev, stream):
            return _clip_copies(grads, out, max_norm, norm_type, eps, ws)
    with _b._on(dev, stream) as s:
        ws, ws_bytes = _workspace(n, ws, dev)
        norm = torch.empty((), dtype=torch.float32, device=dev)
        _b._check(_b.lib().lce_clip_grad_norm(_at(ptrs), _at(sizes), _at(codes), dst, n, kind, max_norm, eps,
                                              norm.data_ptr(), ws.data_ptr(), ws_bytes, s),
                  "lce_clip_grad_norm")
    _b._wrote(grads if out is None else out)
    return norm
