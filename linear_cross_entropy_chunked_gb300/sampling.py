"""Drawing tokens from logits: temperature, top-k, top-p and min-p, by inversion from
given uniform numbers (lce_sample_logits). Argument marshalling only."""
from __future__ import annotations

import math

import torch

from . import _binding as _b


def _setting(name, value, N, dev, dtype):
    """(device pointer or None, value for every row) of one setting."""
    if isinstance(value, torch.Tensor):
        if value.dtype != dtype:
            raise TypeError(f"{name} must be a number or a {dtype} tensor")
        if value.device != dev or value.shape != (N,) or not value.is_contiguous():
            raise ValueError(f"{name} must be a contiguous [N] tensor on the device of Z")
        return value.data_ptr(), 0
    return None, value


def sample_logits(Z, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, tokens=None, logprobs=None,
                  stream=None):
    """One token per row of logits Z [N, V] (bf16, fp16 or fp32, unit column stride, any
    row stride): (tokens int64 [N], logprobs fp32 [N]).

    u [N] fp32 on the device: one uniform number in [0, 1) per row. temperature,
    top_k (0: all), top_p (1: all) and min_p (0: all): numbers, or one value per row in
    a device tensor (fp32; top_k int32). Tokens are ordered by logit, ties by index; top-k
    keeps the first k, top-p of those the shortest prefix that holds the share
    top_p, min-p the tokens at least min_p times as likely as the first; the token is
    the first, by index, at which the kept probability exceeds u, and logprobs the log
    of its share of it. temperature 0 is greedy. -inf and NaN logits are never drawn; a
    row of nothing else gives token -1 and logprob -inf. Weights are rounded to multiples of
    2^-43 of the largest and their sums exact: the same inputs give the same tokens in every
    run. tokens / logprobs: where to write them. V up to 2^20."""
    if not (Z.is_cuda and u.is_cuda):
        raise ValueError("Z and u must be CUDA tensors (there is no CPU path)")
    if Z.dtype not in _b._CE_DTYPES or u.dtype != torch.float32:
        raise TypeError("Z must be bfloat16, float16 or float32 and u float32")
    if Z.dim() != 2 or Z.shape[1] == 0 or (Z.stride(1) != 1 and Z.shape[1] > 1):
        raise ValueError("expected Z[N, V] with unit column stride")
    N, V = Z.shape
    dev = Z.device
    if u.shape != (N,) or not u.is_contiguous() or u.device != dev:
        raise ValueError("u must be a contiguous [N] tensor on the device of Z")
    ld = Z.stride(0) if N > 1 else V
    if ld < V:
        raise ValueError("the rows of Z must not overlap")
    t, t_all = _setting("temperature", temperature, N, dev, torch.float32)
    k, k_all = _setting("top_k", top_k, N, dev, torch.int32)
    p, p_all = _setting("top_p", top_p, N, dev, torch.float32)
    q, q_all = _setting("min_p", min_p, N, dev, torch.float32)
    if not 0.0 <= t_all < math.inf:
        raise ValueError("temperature must be finite and not negative")
    if not 0 <= k_all < math.inf or int(k_all) != k_all:
        raise ValueError("top_k must be a whole number, 0 for all tokens")
    if not 0.0 <= p_all <= 1.0 or not 0.0 <= q_all <= 1.0:
        raise ValueError("top_p and min_p must lie in [0, 1]")
    given = [t for t in (tokens, logprobs) if t is not None]
    with _b._on(dev, stream) as s:
        if tokens is None:
            tokens = torch.empty(N, dtype=torch.int64, device=dev)
        elif tokens.dtype != torch.int64 or tokens.shape != (N,) or not tokens.is_contiguous() \
                or tokens.device != dev:
            raise ValueError("tokens must be a contiguous int64 [N] tensor on the device of Z")
        if logprobs is None:
            logprobs = torch.empty(N, dtype=torch.float32, device=dev)
        elif logprobs.dtype != torch.float32 or logprobs.shape != (N,) or not logprobs.is_contiguous() \
                or logprobs.device != dev:
            raise ValueError("logprobs must be a contiguous float32 [N] tensor on the device of Z")
        _b._check(_b.lib().lce_sample_logits(Z.data_ptr(), _b._CE_DTYPES[Z.dtype], ld, N, V, u.data_ptr(),
                                             t, k, p, q, t_all, min(int(k_all), V), p_all, q_all,
                                             tokens.data_ptr(), logprobs.data_ptr(), s),
                  "lce_sample_logits")
    if given:
        _b._wrote(given)
    return tokens, logprobs
