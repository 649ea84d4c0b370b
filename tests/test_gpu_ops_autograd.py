"""What autograd sees of tensors that the calls write to: a backward pass that saved one refuses to run with
the changed values, as after torch's own in-place operations."""
import pytest
import torch

import linear_cross_entropy_chunked_gb300 as lce

pytestmark = pytest.mark.gpu


def saved_by_a_graph(t):
    """A loss whose backward pass needs t as it is now."""
    w = torch.ones_like(t, requires_grad=True)
    return (w * t).float().sum()


def test_clipping_in_place_is_seen():
    x = torch.randn(1000, device="cuda", requires_grad=True)
    (g,) = torch.autograd.grad((x ** 3).sum(), x, create_graph=True)
    penalty = g.square().sum()                 # its backward pass needs g
    version = g._version
    lce.clip_grad_norm([g], 0.1)
    assert g._version > version
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        penalty.backward()


def test_only_what_is_written_is_seen():
    grads = [torch.randn(n, device="cuda", dtype=t) for n, t in ((70, torch.float32), (300, torch.bfloat16), (0, torch.float16))]
    out = [torch.empty_like(g) for g in grads]
    before = [t._version for t in grads + out]
    lce.grad_norm(grads)
    assert [t._version for t in grads + out] == before
    losses = [saved_by_a_graph(g) for g in grads]
    lce.clip_grad_norm(grads, 0.1, out=out)
    assert [t._version for t in grads] == before[:3]
    assert all(t._version > b for t, b in zip(out, before[3:]))
    for loss in losses:
        loss.backward()                        # the gradients are as they were


def test_outputs_that_are_given_are_seen():
    a, sa = lce.quantize_fp8(torch.randn(4, 128, device="cuda"))
    b, sb = lce.quantize_fp8(torch.randn(64, 128, device="cuda"), tiles=True)
    out = torch.zeros(4, 64, device="cuda")
    loss = saved_by_a_graph(out)
    lce.fp8_matmul(a, sa, b, sb, out=out)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    logprobs, tokens = torch.zeros(4, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    loss, version = saved_by_a_graph(logprobs), tokens._version
    lce.sample_logits(out, torch.rand(4, device="cuda"), logprobs=logprobs, tokens=tokens)
    assert tokens._version > version
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_inference_tensors():
    with torch.inference_mode():
        g = torch.ones(100, device="cuda")
        n = lce.clip_grad_norm([g], 1.0)
    assert n.item() == 10.0 and (g - 0.1).abs().max() < 1e-6
    lce.clip_grad_norm([g, torch.ones(3, device="cuda")], 0.5)   # outside of the mode, beside others
    logprobs = torch.empty(4, device="cuda")
    with torch.inference_mode():
        out = torch.empty(4, dtype=torch.int64, device="cuda")
        lce.sample_logits(torch.randn(4, 50, device="cuda"), torch.rand(4, device="cuda"), tokens=out, logprobs=logprobs)
