"""Widths that are no multiple of 16 bytes: fp8_linear's gradients have padded rows, and clipping takes them
as they come. Tolerances as for clipping dense gradients: 19 * 2^-24 of the norm, 3 roundings more for the
factor, half a step of the type for the product."""
import math

import numpy as np
import pytest
import torch

import linear_cross_entropy_chunked_gb300 as lce
from oracle import ops_oracle

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
NORM_REL = 19 * 2.0 ** -24


def check(norm, got, before, max_norm, norm_type=2.0):
    want, scaled = ops_oracle.clip([b.double().cpu().numpy() for b in before], max_norm, norm_type)
    assert abs(norm.item() - want) <= NORM_REL * want
    for t, w in zip(got, scaled):
        f = torch.finfo(t.dtype)
        err = np.abs(t.detach().double().cpu().numpy() - w)
        assert (err <= (f.eps / 2 + NORM_REL + 3 * 2.0 ** -24) * np.abs(w) + f.smallest_normal * f.eps / 2).all()


def gradients(d, v, dtype, m=70):
    g = torch.Generator().manual_seed(d)
    X, W, dZ = (torch.randn(*s, generator=g).to(DTYPES[dtype]).cuda() for s in ((m, d), (v, d), (m, v)))
    X.requires_grad_()
    W.requires_grad_()
    return X, W, torch.autograd.grad(lce.fp8_linear(X, W), (X, W), dZ)


@pytest.mark.parametrize("norm_type", [2.0, 1.0, math.inf])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("d,v", [(203, 301), (130, 129), (1, 5), (264, 1001)])
def test_gradients_of_the_layer(d, v, dtype, norm_type):
    X, W, grads = gradients(d, v, dtype)
    extra = torch.randn(77, device="cuda")
    before = [g.clone() for g in (*grads, extra)]
    norm = lce.grad_norm([*grads, extra], norm_type)
    limit = 0.5 * norm.item()
    out = [torch.empty_strided(g.shape, g.stride(), dtype=g.dtype, device="cuda") for g in grads] + [torch.empty_like(extra)]
    check(lce.clip_grad_norm([*grads, extra], limit, norm_type, out=out), out, before, limit, norm_type)
    assert all(torch.equal(a, b) for a, b in zip((*grads, extra), before))
    dense = [torch.empty(g.shape, dtype=g.dtype, device="cuda") for g in (*grads, extra)]
    check(lce.clip_grad_norm([*grads, extra], limit, norm_type, out=dense), dense, before, limit, norm_type)
    assert lce.clip_grad_norm([*grads, extra], limit, norm_type).item() == norm.item()
    assert all(torch.equal(a, b) for a, b in zip((*grads, extra), out))
    assert lce.clip_grad_norm([*grads, extra], 1e9, norm_type).item() <= 0.51 * norm.item()   # left as they are
    assert all(torch.equal(a, b) for a, b in zip((*grads, extra), out))


def test_padding_and_versions():
    wide = torch.full((9, 208), 7.0, dtype=torch.bfloat16, device="cuda")
    g = wide[:, :203]
    g.copy_(torch.randn(9, 203))
    before, version = g.clone(), g._version
    check(lce.clip_grad_norm(g, 1.0), [g], [before], 1.0)
    assert (wide[:, 203:] == 7).all() and g._version > version
    x = torch.randn(40, 203, device="cuda", requires_grad=True)
    (dx,) = torch.autograd.grad(x.square().sum(), x, create_graph=True)
    lce.clip_grad_norm([dx, wide[:, :203]], 1.0)           # a gradient that requires one itself


def test_a_step_with_leaves():
    # accumulated into .grad, on another stream, captured
    X, W, grads = gradients(203, 301, "bf16")
    dZ = torch.randn(70, 301, device="cuda").bfloat16()
    lce.fp8_linear(X, W).backward(dZ)
    before = [X.grad.clone(), W.grad.clone()]
    check(lce.clip_grad_norm([X.grad, W.grad], 1.0), [X.grad, W.grad], before, 1.0)
    before = [g.clone() for g in grads]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    norm = lce.clip_grad_norm(grads, 1.0, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    check(norm, grads, before, 1.0)
    graph, static = torch.cuda.CUDAGraph(), [torch.empty_strided(g.shape, g.stride(), dtype=g.dtype, device="cuda") for g in grads]
    with torch.cuda.graph(graph):
        norm = lce.clip_grad_norm(static, 1.0)
    for s, b in zip(static, before):
        s.copy_(b)
    graph.replay()
    check(norm, static, before, 1.0)


def test_refusals():
    _, _, (dX, dW) = gradients(203, 301, "bf16")
    before = [dX.clone(), dW.clone()]
    with pytest.raises(lce.LCEError):
        lce.clip_grad_norm([dX, dX], 1.0)                  # the same tensor twice
    with pytest.raises(lce.LCEError):
        lce.clip_grad_norm([dX, dX[10:20]], 1.0)
    with pytest.raises(lce.LCEError):
        lce.clip_grad_norm([dX, dW], 1.0, out=[dW[:70], torch.empty_like(dW)])  # over another gradient
    with pytest.raises(ValueError):
        lce.clip_grad_norm([dX], 1.0, out=[dX[:60]])
    with pytest.raises(ValueError):
        lce.clip_grad_norm(torch.randn(8, 48, device="cuda")[:, :40], 1.0)      # a slice of something wider
    with pytest.raises(ValueError):
        lce.grad_norm(torch.randn(8, 48, device="cuda")[::2])
    assert torch.equal(dX, before[0]) and torch.equal(dW, before[1])
    assert lce.grad_norm([dX, dX]).item() > 0              # nothing is written
