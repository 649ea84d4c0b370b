"""Losses on answers: the clipped policy loss with a KL term, and the preference loss of paired
log ratios, over the LM head (hidden states and weight) or over logits that the caller holds
(lce_policy_*, lce_preference_*). Argument marshalling only."""
from __future__ import annotations

import ctypes

import torch
from torch.autograd.function import once_differentiable

from . import _binding as _b

DW_BF16 = 32


def _vector(name, t, shape, dtype, dev):
    """Address of a constant of the call (None for None)."""
    if t is None:
        return None
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.device != dev or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {list(shape)} tensor on the device of the other arguments")
    _constant(name, t)
    return t.data_ptr()


def _constant(name, t):
    if t is not None and t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name} is a constant of the loss: detach it")


def _policy_args(N, dev, advantages, old_logprobs, ref_logprobs, weights, clip_low, clip_high, beta, temperature):
    if advantages is None:
        raise TypeError("advantages must be a tensor")
    shape, f32 = (N,), torch.float32
    if beta and ref_logprobs is None:
        raise ValueError("beta needs ref_logprobs")
    return (_vector("advantages", advantages, shape, f32, dev), _vector("old_logprobs", old_logprobs, shape, f32, dev),
            _vector("ref_logprobs", ref_logprobs, shape, f32, dev), _vector("weights", weights, shape, f32, dev),
            clip_low, clip_high, beta, temperature)


def _check_head(H, W, y):
    N, D, V = _b._check_inputs(H, W, y)
    if H.dtype != torch.bfloat16:
        raise TypeError("H and W must be bfloat16 (a row's coefficient has no range that fp16 gradients "
                        "could be scaled by)")
    if W.device != H.device or y.device != H.device:
        raise ValueError("H, W and y must be on one device")
    return N, D, V


def _given(name, t, shape, dtype, dev):
    """A tensor of the caller that the call writes to."""
    if t.dtype != dtype or t.shape != shape or t.device != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} {list(shape)} tensor on the device of the inputs")
    return t


class _Outputs:
    """The outputs of a call: the caller's tensors where there are some, else new ones."""

    def __init__(self, dev):
        self.dev, self.mine = dev, []

    def take(self, name, t, shape, dtype=torch.float32):
        if t is None:
            return torch.empty(shape, dtype=dtype, device=self.dev)
        self.mine.append(_given(name, t, shape, dtype, self.dev))
        return t

    def done(self):
        if self.mine:
            _b._wrote(self.mine)


def _workspace(ws, nbytes, dev):
    if ws is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=dev)
    if ws.device != dev or ws.dtype != torch.uint8 or not ws.is_contiguous() or ws.numel() < nbytes \
            or ws.data_ptr() % 16:
        raise ValueError(f"ws must be a contiguous, 16-byte aligned uint8 tensor of at least {nbytes} bytes")
    return ws


def _loss_shape(reduction, n):
    return (n,) if reduction == "none" else (1,)


def _dloss(dloss, reduction, n, dev):
    return _vector("dloss", None if dloss is None else dloss.detach().reshape(-1), _loss_shape(reduction, n),
                   torch.float32, dev)


def policy_workspace_size(N, D, V, chunk, flags=0, gradient=True):
    out = ctypes.c_size_t(0)
    _b._check(_b.lib().lce_policy_workspace_size(N, D, V, chunk, flags, 1 if gradient else 0, ctypes.byref(out)),
              "lce_policy_workspace_size")
    return out.value


def policy_forward(H, W, y, advantages, old_logprobs=None, ref_logprobs=None, weights=None, clip_low=0.2,
                   clip_high=0.2, beta=0.0, temperature=1.0, chunk: int = 1024,
                   ignore_index: int = _b.IGNORE_INDEX, reduction: str = "mean", loss=None, logprobs=None, ws=None,
                   stream=None):
    """(loss, logprobs) of the policy loss over the head, as policy_fwd_bwd, without gradients."""
    N, D, V = _check_head(H, W, y)
    dev, red = H.device, _b._reduction(reduction)
    args = _policy_args(N, dev, advantages, old_logprobs, ref_logprobs, weights, clip_low, clip_high, beta,
                        temperature)
    with _b._on(dev, stream) as s:
        out = _Outputs(dev)
        loss = out.take("loss", loss, _loss_shape(reduction, N))
        logprobs = out.take("logprobs", logprobs, (N,))
        ws = _workspace(ws, policy_workspace_size(N, D, V, chunk, gradient=False), dev)
        _b._check(_b.lib().lce_policy_forward(
            H.data_ptr(), W.data_ptr(), y.data_ptr(), *args, N, D, V, ignore_index, chunk, red, loss.data_ptr(),
            logprobs.data_ptr(), ws.data_ptr(), ws.numel(), s), "lce_policy_forward")
        out.done()
    return loss, logprobs


def _gradients(out, H, W, dH, dW, accumulate, compute_dW, low_memory, dW_dtype):
    if dW_dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("dW_dtype must be float32 or bfloat16")
    flags = _b._acc_flags(accumulate, dH, dW, compute_dW) | (_b.LOW_MEMORY if low_memory else 0)
    if compute_dW and dW_dtype == torch.bfloat16:
        flags |= DW_BF16
    dH = out.take("dH", dH, tuple(H.shape), H.dtype)
    return flags, dH, out.take("dW", dW, tuple(W.shape), dW_dtype) if compute_dW else None


def policy_fwd_bwd(H, W, y, advantages, old_logprobs=None, ref_logprobs=None, weights=None, clip_low=0.2,
                   clip_high=0.2, beta=0.0, temperature=1.0, dloss=None, chunk: int = 1024,
                   ignore_index: int = _b.IGNORE_INDEX, reduction: str = "mean", loss=None, logprobs=None, dH=None,
                   dW=None, ws=None, stream=None, accumulate=(), compute_dW: bool = True, low_memory: bool = False,
                   dW_dtype=torch.float32):
    """The clipped policy loss over the head, with its gradients: (loss, logprobs, dH, dW).

    H [N, D] and W [V, D] bf16, y [N] the drawn tokens (ignore_index: the row does not count), and
    fp32 [N]: advantages, old_logprobs (None: the tokens come from this very policy),
    ref_logprobs (of the reference model; needed where beta is not 0), weights (None: 1). With
    logp the token's log probability at the temperature and r = exp(logp - old):
        loss = w (-min(r A, clamp(r, 1 - clip_low, 1 + clip_high) A) + beta (e^d - 1 - d)),  d = ref - logp
    reduction: the mean over the counting rows, "sum" (a mean over sequences has its weights
    1 / (tokens * sequences)), or "none" (loss [N]; dloss [N]). logprobs [N]: logp, 0 for rows that
    do not count. dH bf16, dW fp32 (or bf16 by dW_dtype, where the rows fill one buffer and dW is not added
    to). chunk: the memory / speed knob: a buffer of 2 chunk rows of logits (low_memory: chunk rows).
    The rest as for lce_fwd_bwd."""
    N, D, V = _check_head(H, W, y)
    dev, red = H.device, _b._reduction(reduction)
    args = _policy_args(N, dev, advantages, old_logprobs, ref_logprobs, weights, clip_low, clip_high, beta,
                        temperature)
    d = _dloss(dloss, reduction, N, dev)
    with _b._on(dev, stream) as s:
        out = _Outputs(dev)
        loss = out.take("loss", loss, _loss_shape(reduction, N))
        logprobs = out.take("logprobs", logprobs, (N,))
        flags, dH, dW = _gradients(out, H, W, dH, dW, accumulate, compute_dW, low_memory, dW_dtype)
        ws = _workspace(ws, policy_workspace_size(N, D, V, chunk, flags), dev)
        _b._check(_b.lib().lce_policy_fwd_bwd(
            H.data_ptr(), W.data_ptr(), y.data_ptr(), *args, d, N, D, V, ignore_index, chunk, red, flags,
            loss.data_ptr(), logprobs.data_ptr(), dH.data_ptr(), None if dW is None else dW.data_ptr(),
            ws.data_ptr(), ws.numel(), s), "lce_policy_fwd_bwd")
        out.done()
    return loss, logprobs, dH, dW


def preference_workspace_size(N, D, V, chunk, pairs, flags=0, gradient=True):
    out = ctypes.c_size_t(0)
    _b._check(_b.lib().lce_preference_workspace_size(N, D, V, chunk, pairs, flags, 1 if gradient else 0,
                                                     ctypes.byref(out)), "lce_preference_workspace_size")
    return out.value


def _pairs(offsets, dev):
    if offsets.dim() != 1 or offsets.shape[0] < 3 or offsets.shape[0] % 2 == 0:
        raise ValueError("offsets must be [2 pairs + 1]: the chosen sequences, then the rejected ones")
    _vector("offsets", offsets, (offsets.shape[0],), torch.int64, dev)
    return offsets.shape[0] // 2


def preference_fwd_bwd(H, W, y, offsets, ref_logprobs=None, beta=0.1, label_smoothing=0.0, average: bool = False,
                       dloss=None, chunk: int = 1024, ignore_index: int = _b.IGNORE_INDEX, reduction: str = "mean",
                       loss=None, seq_logprobs=None, dH=None, dW=None, ws=None, stream=None, accumulate=(),
                       gradient: bool = True, compute_dW: bool = True, low_memory: bool = False,
                       dW_dtype=torch.float32):
    """The preference loss of paired log ratios over the head, with its gradients: (loss,
    seq_logprobs, dH, dW).

    H [N, D] and W [V, D] bf16, y [N] (ignore_index: the row does not count). The rows of sequence s are
    offsets[s] .. offsets[s + 1] - 1 (int64 [2 pairs + 1] on the device); sequence k is the
    chosen one of pair k, sequence pairs + k the rejected one. With L the sum (average: the mean) of
    a sequence's log probabilities and R the reference's (ref_logprobs fp32 [2 pairs], None: 0):
        m = beta ((L_c - R_c) - (L_r - R_r))
        loss = -((1 - label_smoothing) log sigmoid(m) + label_smoothing log sigmoid(-m))
    reduction: the mean over the pairs, "sum", or "none" (loss [pairs]; dloss [pairs]).
    seq_logprobs [2 pairs]: L; a reference model's, from a call with gradient=False (dH and dW are None
    then), is the ref_logprobs of this one. Up to 2 chunk counting rows no logits are computed twice: a
    larger chunk is faster and takes more workspace. Rows outside the sequences add nothing."""
    N, D, V = _check_head(H, W, y)
    dev, red = H.device, _b._reduction(reduction)
    P = _pairs(offsets, dev)
    ref = _vector("ref_logprobs", ref_logprobs, (2 * P,), torch.float32, dev)
    d = _dloss(dloss, reduction, P, dev)
    with _b._on(dev, stream) as s:
        out = _Outputs(dev)
        loss = out.take("loss", loss, _loss_shape(reduction, P))
        seq_logprobs = out.take("seq_logprobs", seq_logprobs, (2 * P,))
        if gradient:
            flags, dH, dW = _gradients(out, H, W, dH, dW, accumulate, compute_dW, low_memory, dW_dtype)
        elif dH is not None or dW is not None or accumulate:
            raise ValueError("no gradients were asked for")
        else:
            flags = _b.LOW_MEMORY if low_memory else 0
        ws = _workspace(ws, preference_workspace_size(N, D, V, chunk, P, flags, gradient), dev)
        _b._check(_b.lib().lce_preference_fwd_bwd(
            H.data_ptr(), W.data_ptr(), y.data_ptr(), offsets.data_ptr(), P, ref, beta, label_smoothing,
            1 if average else 0, d, N, D, V, ignore_index, chunk, red, flags, loss.data_ptr(),
            seq_logprobs.data_ptr(), None if dH is None else dH.data_ptr(), None if dW is None else dW.data_ptr(),
            ws.data_ptr(), ws.numel(), s), "lce_preference_fwd_bwd")
        out.done()
    return loss, seq_logprobs, dH, dW


def _scaled(src, scale, dtype, s):
    """src * scale[0] in dtype, rounded once."""
    out = torch.empty(src.shape, dtype=dtype, device=src.device)
    _b._check(_b.lib().lce_scale(src.data_ptr(), _b._CE_DTYPES[src.dtype], scale.data_ptr(), src.numel(),
                                 out.data_ptr(), _b._CE_DTYPES[dtype], s), "lce_scale")
    return out


def _scale_in_place(t, scale, s):
    _b._check(_b.lib().lce_scale(t.data_ptr(), _b._CE_DTYPES[t.dtype], scale.data_ptr(), t.numel(), t.data_ptr(),
                                 _b._CE_DTYPES[t.dtype], s), "lce_scale")
    return t


class AnswerLossFunction(torch.autograd.Function):
    """A loss on answers over the head. The forward forms the gradients for an upstream gradient
    of 1 (fwd_bwd), dH in H's dtype and dW in the one that it is told; the backward scales them, which
    the loss is linear in, in place (nothing is read or written where the upstream gradient is 1; one that is no
    power of two rounds bf16 gradients once more, an fp32 dW only then), and hands them over. A second backward
    through the same graph forms them again, and so does a backward that is captured without its forward (each
    replay would scale them once more; captured in a graph of its own behind that of its forward, it is replayed once
    for each replay of that). A W without requires_grad is frozen (no dW work). The log probabilities beside the loss
    carry no gradient."""

    @staticmethod
    def forward(ctx, H, W, fwd_bwd, dW_dtype, *constants):
        train = ctx.needs_input_grad[1]
        how = {"compute_dW": train, "dW_dtype": dW_dtype if train else torch.float32}
        loss, logprobs, *gradients = fwd_bwd(H, W, *constants, **how)
        ctx.gradients = [gradients]   # (taken once, whichever of two threads comes first)
        ctx.save_for_backward(H, W, *constants)
        ctx.fwd_bwd, ctx.how = fwd_bwd, how
        ctx.captured = H.is_cuda and torch.cuda.is_current_stream_capturing()
        ctx.mark_non_differentiable(logprobs)
        return loss.view(()), logprobs

    @staticmethod
    @once_differentiable
    def backward(ctx, g, _):
        tensors = ctx.saved_tensors   # (that none was written to since is checked here)
        g = g.to(torch.float32).contiguous()
        with _b._on(tensors[0].device, None) as s:
            mine = None
            if torch.cuda.is_current_stream_capturing() == ctx.captured:
                try:
                    mine = ctx.gradients.pop()
                except IndexError:
                    pass
            if mine is None:
                _, _, dH, dW = ctx.fwd_bwd(*tensors, dloss=g, **ctx.how)
                dW = dW if dW is None or dW.dtype == tensors[1].dtype else dW.to(tensors[1].dtype)
            else:
                dH, dW = mine
                if ctx.needs_input_grad[0]:
                    _scale_in_place(dH, g, s)
                if dW is not None:
                    dW = _scale_in_place(dW, g, s) if dW.dtype == tensors[1].dtype else \
                        _scaled(dW, g, tensors[1].dtype, s)
        return (dH if ctx.needs_input_grad[0] else None, dW, None, None) + (None,) * (len(tensors) - 2)


def _dW_dtype(dtype, H, chunk, low_memory):
    """bf16 by default where the rows fill one chunk buffer, so that dW is one contraction: a third of the memory traffic."""
    one = H.shape[0] <= (1 if low_memory else 2) * chunk
    if dtype is None:
        return torch.bfloat16 if one else torch.float32
    if dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("dW_dtype must be float32 or bfloat16")
    if dtype == torch.bfloat16 and not one:
        raise ValueError("dW_dtype bfloat16 needs rows that fill one chunk buffer")
    return dtype


def _summed(what, reduction):
    if reduction not in ("mean", "sum"):
        raise ValueError(f"{what} supports reduction 'mean' or 'sum' (a reduction of 'none' needs the upstream "
                         f"gradient before the backward: call {what.replace('linear_', '').replace('_loss', '')}_fwd_bwd)")


def linear_policy_loss(H, W, y, advantages, old_logprobs=None, ref_logprobs=None, weights=None, clip_low=0.2,
                       clip_high=0.2, beta=0.0, temperature=1.0, chunk: int = 1024,
                       ignore_index: int = _b.IGNORE_INDEX, reduction: str = "mean", low_memory: bool = False,
                       dW_dtype=None):
    """(loss, logprobs): the clipped policy loss with a KL term over the head (policy_fwd_bwd says
    what the arguments are), differentiable in H and W for the reductions mean and sum. The
    logprobs [N] are those of the policy as it is now, and carry no gradient. A W with
    requires_grad False is frozen. dW_dtype: in what the weight's gradient is kept until the upstream gradient is
    known; None: bf16 where the rows fill one buffer, which is fastest; float32: an upstream gradient of 1 / 3 (a loss over
    three micro-batches) does not round it a second time."""
    _summed("linear_policy_loss", reduction)
    how = {"old_logprobs": old_logprobs, "ref_logprobs": ref_logprobs, "weights": weights, "clip_low": clip_low,
           "clip_high": clip_high, "beta": beta, "temperature": temperature, "chunk": chunk,
           "ignore_index": ignore_index, "reduction": reduction}
    if not (torch.is_grad_enabled() and (H.requires_grad or W.requires_grad)):
        loss, logprobs = policy_forward(H, W, y, advantages, **how)
        return loss.view(()), logprobs
    _constant("advantages", advantages)
    for name in ("old_logprobs", "ref_logprobs", "weights"):
        _constant(name, how.pop(name))
    return AnswerLossFunction.apply(
        H, W, lambda *t, **more: policy_fwd_bwd(*t, low_memory=low_memory, **how, **more),
        _dW_dtype(dW_dtype, H, chunk, low_memory), y, advantages, old_logprobs, ref_logprobs, weights)


def linear_preference_loss(H, W, y, offsets, ref_logprobs=None, beta=0.1, label_smoothing=0.0,
                           average: bool = False, chunk: int = 1024, ignore_index: int = _b.IGNORE_INDEX,
                           reduction: str = "mean", low_memory: bool = False, dW_dtype=None):
    """(loss, seq_logprobs): the preference loss of paired log ratios over the head
    (preference_fwd_bwd says what the arguments are), differentiable in H and W for the
    reductions mean and sum. seq_logprobs [2 pairs] carry no gradient; without gradients the call
    gives a reference model's, which are this one's ref_logprobs. A W with requires_grad False is frozen.
    dW_dtype: as for linear_policy_loss."""
    _summed("linear_preference_loss", reduction)
    how = {"ref_logprobs": ref_logprobs, "beta": beta, "label_smoothing": label_smoothing, "average": average,
           "chunk": chunk, "ignore_index": ignore_index, "reduction": reduction, "low_memory": low_memory}
    if not (torch.is_grad_enabled() and (H.requires_grad or W.requires_grad)):
        loss, seq, _, _ = preference_fwd_bwd(H, W, y, offsets, gradient=False, **how)
        return loss.view(()), seq
    _constant("ref_logprobs", how.pop("ref_logprobs"))
    return AnswerLossFunction.apply(H, W, lambda *t, **more: preference_fwd_bwd(*t, **how, **more),
                                    _dW_dtype(dW_dtype, H, chunk, low_memory), y, offsets, ref_logprobs)


def _check_logits(Z, y):
    if not (Z.is_cuda and y.is_cuda):
        raise ValueError("Z and y must be CUDA tensors (there is no CPU path)")
    if Z.dtype not in _b._CE_DTYPES or y.dtype != torch.int64:
        raise TypeError("Z must be bfloat16, float16 or float32 and y int64")
    if Z.dim() != 2 or Z.shape[1] == 0 or (Z.stride(1) != 1 and Z.shape[1] > 1):
        raise ValueError("expected Z[N, V] with unit column stride")
    N, V = Z.shape
    if y.shape != (N,) or not y.is_contiguous() or y.device != Z.device:
        raise ValueError("y must be a contiguous [N] tensor on the device of Z")
    ld = Z.stride(0) if N > 1 else V
    if ld < V:
        raise ValueError("the rows of Z must not overlap")
    return N, V, ld


def _gradient_of_logits(Z, ld, grad, inplace):
    """dZ: Z itself, or a tensor whose rows lie as Z's do (row stride, address modulo 16)."""
    if not grad:
        if inplace:
            raise ValueError("no gradient was asked for")
        return None
    if inplace:
        if Z.requires_grad and torch.is_grad_enabled():
            raise ValueError("the gradient cannot be written over logits that require one")
        return Z
    at = Z.data_ptr() % 16 // Z.element_size()
    N, V = Z.shape
    if at == 0:
        return torch.empty_strided((N, V), (ld, 1), dtype=Z.dtype, device=Z.device)
    buf = torch.empty(at + max(0, (N - 1) * ld + V) if N else 0, dtype=Z.dtype, device=Z.device)
    return torch.as_strided(buf, (N, V), (ld, 1), at)


def policy_logits(Z, y, advantages, old_logprobs=None, ref_logprobs=None, weights=None, clip_low=0.2, clip_high=0.2,
                  beta=0.0, temperature=1.0, dloss=None, ignore_index: int = _b.IGNORE_INDEX,
                  reduction: str = "mean", grad: bool = True, inplace: bool = False, loss=None, logprobs=None,
                  ws=None, stream=None):
    """The policy loss of policy_fwd_bwd over precomputed logits Z [N, V] (bf16, fp16 or fp32,
    unit column stride, any row stride): (loss, logprobs, dZ). dZ is None when grad is False; with inplace=True it
    overwrites Z."""
    N, V, ld = _check_logits(Z, y)
    dev, red = Z.device, _b._reduction(reduction)
    args = _policy_args(N, dev, advantages, old_logprobs, ref_logprobs, weights, clip_low, clip_high, beta,
                        temperature)
    d = _dloss(dloss, reduction, N, dev)
    with _b._on(dev, stream) as s:
        out = _Outputs(dev)
        loss = out.take("loss", loss, _loss_shape(reduction, N))
        logprobs = out.take("logprobs", logprobs, (N,))
        dZ = _gradient_of_logits(Z, ld, grad, inplace)
        ws = _workspace(ws, 1024 + (4 * max(N, 1) + 1023) // 1024 * 1024, dev)
        _b._check(_b.lib().lce_policy_logits(
            Z.data_ptr(), _b._CE_DTYPES[Z.dtype], ld, y.data_ptr(), *args, d, N, V, ignore_index, red,
            loss.data_ptr(), logprobs.data_ptr(), None if dZ is None else dZ.data_ptr(), ws.data_ptr(), ws.numel(),
            s), "lce_policy_logits")
        if inplace:
            out.mine.append(Z)
        out.done()
    return loss, logprobs, dZ


def preference_logits(Z, y, offsets, ref_logprobs=None, beta=0.1, label_smoothing=0.0, average: bool = False,
                      dloss=None, ignore_index: int = _b.IGNORE_INDEX, reduction: str = "mean", grad: bool = True,
                      inplace: bool = False, loss=None, seq_logprobs=None, ws=None, stream=None):
    """The preference loss of preference_fwd_bwd over precomputed logits Z [N, V] (bf16, fp16 or
    fp32, unit column stride, any row stride): (loss, seq_logprobs, dZ). dZ is None when grad is
    False; with inplace=True it overwrites Z."""
    N, V, ld = _check_logits(Z, y)
    dev, red = Z.device, _b._reduction(reduction)
    P = _pairs(offsets, dev)
    ref = _vector("ref_logprobs", ref_logprobs, (2 * P,), torch.float32, dev)
    d = _dloss(dloss, reduction, P, dev)
    with _b._on(dev, stream) as s:
        out = _Outputs(dev)
        loss = out.take("loss", loss, _loss_shape(reduction, P))
        seq_logprobs = out.take("seq_logprobs", seq_logprobs, (2 * P,))
        dZ = _gradient_of_logits(Z, ld, grad, inplace)
        nbytes = ctypes.c_size_t(0)
        _b._check(_b.lib().lce_preference_logits_workspace_size(N, P, ctypes.byref(nbytes)),
                  "lce_preference_logits_workspace_size")
        ws = _workspace(ws, nbytes.value, dev)
        _b._check(_b.lib().lce_preference_logits(
            Z.data_ptr(), _b._CE_DTYPES[Z.dtype], ld, y.data_ptr(), offsets.data_ptr(), P, ref, beta,
            label_smoothing, 1 if average else 0, d, N, V, ignore_index, red, loss.data_ptr(),
            seq_logprobs.data_ptr(), None if dZ is None else dZ.data_ptr(), ws.data_ptr(), ws.numel(), s),
            "lce_preference_logits")
        if inplace:
            out.mine.append(Z)
        out.done()
    return loss, seq_logprobs, dZ
