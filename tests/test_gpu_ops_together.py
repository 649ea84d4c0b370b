"""Sampling, the 8-bit linear layer and gradient clipping as they are used together, and the Python calls'
refusals of device tensors that do not fit."""
import threading

import numpy as np
import pytest
import torch

import linear_cross_entropy_chunked_gb300 as lce
from oracle import lce_oracle, ops_oracle

pytestmark = pytest.mark.gpu


def inputs(m, v, d, seed, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    X = (torch.randn(m, d, generator=g)).to(dtype).cuda()
    W = (torch.randn(v, d, generator=g) * 0.05).to(dtype).cuda()
    return X, W, torch.randint(0, v, (m,), generator=g).cuda(), torch.rand(m, generator=g).cuda()


def full(x, tiles=False):
    q, s = ops_oracle.quantize_fp8(x.detach().double().cpu().numpy(), tiles)
    return torch.from_numpy(ops_oracle.dequantize_fp8(q, s))


@pytest.mark.parametrize("m,v,d", [(70, 1001, 200), (200, 3000, 384)])
def test_a_training_step(m, v, d):
    # logits in 8 bits, cross-entropy over them, both gradients in 8 bits, clipped together
    X, W, y, _ = inputs(m, v, d, m)
    X.requires_grad_()
    W.requires_grad_()
    Z = lce.fp8_linear(X, W)
    loss, lse, dZ = lce.ce_logits(Z.detach(), y)
    dX, dW = torch.autograd.grad(Z, (X, W), dZ)
    before = [dX.clone(), dW.clone()]
    norm = lce.clip_grad_norm([dX, dW], 0.01)
    # the loss of the logits as they are, in fp64
    ref = lce_oracle.ce_from_logits(Z.detach().cpu(), y.cpu())
    assert abs(loss.item() - ref["loss"]) <= 1e-3 * abs(ref["loss"])
    # the gradients of the formulas, from the dZ that was handed on; a product's error is at most
    # (128 + blocks + 4) 2^-23 of the sum of magnitudes, and half a bf16 step
    z, zt = full(dZ), full(dZ.t())
    want = z @ full(W, True), zt @ full(X.t()).t()
    mass = z.abs() @ full(W, True).abs(), zt.abs() @ full(X.t()).t().abs()
    for got, w, s, k in zip(before, want, mass, (v, m)):
        bound = (132 + -(-k // 128)) * 2.0 ** -23 * s
        err = (got.double().cpu() - w).abs()
        assert (err <= bound + 2.0 ** -8 * (w.abs() + bound)).all()
    n, scaled = ops_oracle.clip([b.double().cpu().numpy() for b in before], 0.01)
    assert abs(norm.item() - n) <= 19 * 2.0 ** -24 * n
    for got, s in zip((dX, dW), scaled):
        assert (np.abs(got.double().cpu().numpy() - s) <= (2.0 ** -8 + 22 * 2.0 ** -24) * np.abs(s) + 1e-40).all()


def test_a_decoding_step_captured():
    # RMSNorm, 8-bit head, sampling with settings per request; replays follow new inputs
    m, v, d = 9, 5003, 256
    X, W, _, u = inputs(m, v, d, 1)
    gamma = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    w8 = lce.fp8_weight(W, transpose=False)
    t = torch.tensor([0.0, 0.7, 1.0] * 3, device="cuda")
    k = torch.tensor([0, 50, 0] * 3, dtype=torch.int32, device="cuda")
    p = torch.tensor([1.0, 0.9, 0.8] * 3, device="cuda")

    def step():
        with torch.no_grad():
            H = lce.rmsnorm_forward(X, gamma)
            Z = lce.fp8_linear(H, w8)
            return (Z,) + lce.sample_logits(Z, u, temperature=t, top_k=k, top_p=p)
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Z, tokens, logprobs = step()
    for seed in (2, 3, 4):
        X2, _, _, u2 = inputs(m, v, d, seed)
        X.copy_(X2)
        u.copy_(u2)
        graph.replay()
        eager = step()
        assert all(torch.equal(a, b) for a, b in zip((Z, tokens, logprobs), eager))
        ref = ops_oracle.sample(Z.double().cpu().numpy(), u.double().cpu().numpy(), t.cpu().numpy(), k.cpu().numpy(),
                                p.cpu().numpy())
        np.testing.assert_array_equal(tokens.cpu().numpy(), ref["tokens"])


def test_backward_captured_beside_an_eager_graph():
    # (torch cannot capture a backward pass into leaves of which an eager graph lives, whatever the
    # operation: the captured one gets leaves of its own over the same memory)
    X, W, _, _ = inputs(33, 700, 128, 5)
    X.requires_grad_()
    W.requires_grad_()
    dZ = torch.randn(33, 700, device="cuda").bfloat16()
    eager = lce.fp8_linear(X, W)                       # lives on while the other is captured
    want = torch.autograd.grad(lce.fp8_linear(X, W), (X, W), dZ)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x, w = X.detach().requires_grad_(), W.detach().requires_grad_()
        got = torch.autograd.grad(lce.fp8_linear(x, w), (x, w), dZ)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(torch.equal(a, b) for a, b in zip(torch.autograd.grad(eager, (X, W), dZ), want))
    with torch.no_grad():
        X.copy_(inputs(33, 700, 128, 6)[0])
    graph.replay()
    want = torch.autograd.grad(lce.fp8_linear(X, W), (X, W), dZ)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_threads_on_two_streams():
    X, W, _, u = inputs(40, 3001, 256, 6)
    w8 = lce.fp8_weight(W)
    with torch.no_grad():
        Z = lce.fp8_linear(X, w8)
    want = (Z, *lce.sample_logits(Z, u, top_k=20, top_p=0.9), lce.grad_norm([X, W]))
    torch.cuda.synchronize()
    failures = []

    def work():
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream), torch.no_grad():
                for _ in range(20):
                    z = lce.fp8_linear(X, w8)
                    got = (z, *lce.sample_logits(z, u, top_k=20, top_p=0.9), lce.grad_norm([X, W]))
                    stream.synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want)):
                        failures.append("another result")
        except Exception as e:  # noqa: BLE001
            failures.append(repr(e))
    threads = [threading.Thread(target=work) for _ in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not failures, failures


def test_sampling_refusals():
    Z, u = torch.randn(4, 100, device="cuda"), torch.rand(4, device="cuda")
    for bad in (dict(temperature=-1.0), dict(temperature=float("inf")), dict(temperature=float("nan")),
                dict(top_k=-1), dict(top_k=1.5), dict(top_p=1.5), dict(top_p=-0.1), dict(min_p=2.0),
                dict(temperature=torch.ones(3, device="cuda")), dict(temperature=torch.ones(4)),
                dict(top_p=torch.ones(8, device="cuda")[::2]),
                dict(tokens=torch.empty(4, dtype=torch.int32, device="cuda")),
                dict(logprobs=torch.empty(5, device="cuda"))):
        with pytest.raises(ValueError):
            lce.sample_logits(Z, u, **bad)
    for bad in (dict(temperature=torch.ones(4, dtype=torch.float64, device="cuda")),
                dict(top_k=torch.ones(4, dtype=torch.int64, device="cuda"))):
        with pytest.raises(TypeError):
            lce.sample_logits(Z, u, **bad)
    with pytest.raises(TypeError):
        lce.sample_logits(Z.double(), u)
    with pytest.raises(TypeError):
        lce.sample_logits(Z, u.double())
    for z in (Z.t(), Z[:, ::2], Z[0], torch.randn(100, device="cuda").expand(4, 100), Z[:, :0]):
        with pytest.raises(ValueError):
            lce.sample_logits(z, u)
    with pytest.raises(ValueError):
        lce.sample_logits(Z, u[:3])


def test_fp8_refusals():
    X = torch.randn(4, 100, device="cuda", dtype=torch.bfloat16)
    W = torch.randn(50, 100, device="cuda", dtype=torch.bfloat16)
    w8 = lce.fp8_weight(W, transpose=False)
    q, s = lce.quantize_fp8(X)
    for x in (X.t(), X[0], X[:, ::2], X.expand(2, 4, 100)):
        with pytest.raises(ValueError):
            lce.quantize_fp8(x)
    with pytest.raises(TypeError):
        lce.quantize_fp8(X.double())
    with pytest.raises(ValueError):
        lce.fp8_linear(X[:, :96], W)
    with pytest.raises(ValueError):                       # no transpose for the gradient
        lce.fp8_linear(X.clone().requires_grad_(), w8)
    with pytest.raises(TypeError):
        lce.fp8_linear(X, W.double())
    with pytest.raises(ValueError):
        lce.fp8_matmul(q, s.t(), w8.q, w8.scale)
    with pytest.raises(ValueError):                       # A's scales per tile
        lce.fp8_matmul(*lce.quantize_fp8(X.repeat(2, 1), tiles=True), w8.q, w8.scale)
    with pytest.raises(TypeError):
        lce.fp8_matmul(X, s, w8.q, w8.scale)
    with pytest.raises(ValueError):                       # rows that do not start on 16 bytes
        lce.fp8_matmul(q.contiguous(), s, w8.q, w8.scale)
    with pytest.raises(ValueError):
        lce.fp8_matmul(q, s, w8.q, w8.scale, out=torch.empty(4, 50, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        lce.fp8_matmul(q, s, w8.q, w8.scale, out=torch.empty(4, 48, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        lce.fp8_matmul(q, s, w8.q, w8.scale, out_dtype=torch.float64)
    with pytest.raises(ValueError):
        lce.fp8_matmul(q, s, w8.q, w8.scale, ws=torch.empty(100, dtype=torch.uint8, device="cuda"))
    # scales with other strides are the same scales
    want = lce.fp8_matmul(q, s, w8.q, w8.scale)
    assert torch.equal(want, lce.fp8_matmul(q, s.contiguous(), w8.q, w8.scale.t().contiguous().t()))


def test_clip_refusals():
    g = torch.randn(100, device="cuda")
    with pytest.raises(lce.LCEError):
        lce.clip_grad_norm([g, g], 1.0)                    # the same tensor twice
    with pytest.raises(lce.LCEError):
        lce.clip_grad_norm([g[:60], g[50:]], 1.0)
    with pytest.raises(lce.LCEError):
        lce.clip_grad_norm([g[:50], g[50:]], 1.0, out=[torch.empty(50, device="cuda"), g[:50]])
    assert lce.grad_norm([g, g]).item() > 0               # nothing is written
    with pytest.raises(ValueError):
        lce.clip_grad_norm([g], 1.0, out=[])
    with pytest.raises(ValueError):
        lce.clip_grad_norm([g], 1.0, out=[g[:50]])
    with pytest.raises(ValueError):
        lce.clip_grad_norm([g], 1.0, out=[g.bfloat16()])
    with pytest.raises(ValueError):
        lce.clip_grad_norm([g], 1.0, norm_type=0.5)
    with pytest.raises(ValueError):
        lce.clip_grad_norm([g], 1.0, eps=-1.0)
    with pytest.raises(ValueError):
        lce.clip_grad_norm([g, g.cpu()], 1.0)
    with pytest.raises(TypeError):
        lce.clip_grad_norm([g.double()], 1.0)
    with pytest.raises(lce.LCEError):
        lce.grad_norm(g, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))


def test_refused_top_k_without_end():
    Z, u = torch.zeros(2, 10, device="cuda"), torch.zeros(2, device="cuda")
    for k in (float("inf"), float("nan"), -1, 2.5):
        with pytest.raises(ValueError):
            lce.sample_logits(Z, u, top_k=k)
