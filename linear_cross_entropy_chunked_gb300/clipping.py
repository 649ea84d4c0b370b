"""The global norm of a list of gradients, and clipping by it (lce_grad_norm,
lce_clip_grad_norm). Argument marshalling only."""
from __future__ import annotations

import ctypes
import math

import torch

from . import _binding as _b

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


def _tensors(grads, what):
    grads = [grads] if isinstance(grads, torch.Tensor) else list(grads)
    if not grads:
        raise ValueError(f"{what} is empty")
    dev = grads[0].device
    for g in grads:
        if not g.is_cuda:
            raise ValueError(f"{what} must be CUDA tensors (there is no CPU path)")
        if g.dtype not in _b._CE_DTYPES:
            raise TypeError(f"{what} must be bfloat16, float16 or float32")
        if g.device != dev:
            raise ValueError(f"{what} must be on one device")
        if not _dense(g):
            raise ValueError(f"{what} must fill their memory (contiguous or permuted, no gaps)")
    return grads, dev


def _kind(norm_type):
    kind = NORM_KINDS.get(float(norm_type))
    if kind is None:
        raise ValueError("norm_type must be 1, 2 or inf")
    return kind


def _arrays(grads):
    n = len(grads)
    return ((ctypes.c_void_p * n)(*[g.data_ptr() for g in grads]),
            (ctypes.c_int64 * n)(*[g.numel() for g in grads]),
            (ctypes.c_int32 * n)(*[_b._CE_DTYPES[g.dtype] for g in grads]), n)


def _workspace(n, ws, dev):
    if ws is not None:
        if ws.device != dev or not ws.is_contiguous():
            raise ValueError("ws must be a contiguous tensor on the gradients' device")
        return ws, ws.numel() * ws.element_size()
    nbytes = ctypes.c_size_t(0)
    _b._check(_b.lib().lce_grad_norm_workspace_size(n, ctypes.byref(nbytes)), "lce_grad_norm_workspace_size")
    return torch.empty(nbytes.value, dtype=torch.uint8, device=dev), nbytes.value


def grad_norm(grads, norm_type=2.0, ws=None, stream=None):
    """The norm (1, 2 or inf) over all values of the gradients, a tensor or a list of
    tensors (bf16, fp16 and fp32 may be mixed): a device fp32 scalar."""
    kind = _kind(norm_type)
    grads, dev = _tensors(grads, "grads")
    src, sizes, dtypes, n = _arrays(grads)
    with _b._on(dev, stream) as s:
        ws, ws_bytes = _workspace(n, ws, dev)
        norm = torch.empty((), dtype=torch.float32, device=dev)
        _b._check(_b.lib().lce_grad_norm(src, sizes, dtypes, n, kind, norm.data_ptr(), ws.data_ptr(),
                                         ws_bytes, s), "lce_grad_norm")
    return norm


def clip_grad_norm(grads, max_norm, norm_type=2.0, eps=1e-6, out=None, ws=None, stream=None):
    """Scales the gradients (a tensor or a list, bf16, fp16 and fp32 may be mixed) by
    min(1, max_norm / (norm + eps)), in place or into the tensors `out` of the same
    dtypes and layouts, and returns their norm (1, 2 or inf over all values; a device fp32
    scalar; the host does not wait). The factor is formed on the device: gradients
    whose norm is below max_norm stay as they are and are not written in place. A norm
    that is NaN (infinite) makes the factor NaN (0)."""
    kind = _kind(norm_type)
    max_norm, eps = float(max_norm), float(eps)
    if not max_norm >= 0.0 or not 0.0 <= eps < math.inf:
        raise ValueError("max_norm must not be negative, and eps finite and not negative")
    grads, dev = _tensors(grads, "grads")
    src, sizes, dtypes, n = _arrays(grads)
    dst = None
    if out is not None:
        out, out_dev = _tensors(out, "out")
        if len(out) != n or out_dev != dev or any(
                o.dtype != g.dtype or o.shape != g.shape or o.stride() != g.stride()
                for o, g in zip(out, grads)):
            raise ValueError("out must match the gradients in number, device, dtypes, shapes and strides")
        dst = (ctypes.c_void_p * n)(*[o.data_ptr() for o in out])
    with _b._on(dev, stream) as s:
        ws, ws_bytes = _workspace(n, ws, dev)
        norm = torch.empty((), dtype=torch.float32, device=dev)
        _b._check(_b.lib().lce_clip_grad_norm(src, sizes, dtypes, dst, n, kind, max_norm, eps,
                                              norm.data_ptr(), ws.data_ptr(), ws_bytes, s),
                  "lce_clip_grad_norm")
    return norm
