"""The quantisation and the product in one call where the product is shared out along K: the parts' sums
and the operand that is being read lie in one workspace.

Tolerances as for the products: with S = sum over k of |sa a sb b|, at most (128 + blocks + 4) steps of
2^-23 of S, 8 more for the sums of up to 8 parts, and half a step of the output's type."""
import ctypes

import pytest
import torch

import linear_cross_entropy_chunked_gb300 as lce

pytestmark = pytest.mark.gpu


def make(m, n, k):
    g = torch.Generator(device="cuda").manual_seed(m + n + k)
    X = torch.randn(m, k, device="cuda", generator=g) * torch.exp(0.5 * torch.randn(m, 1, device="cuda", generator=g))
    W = torch.randn(n, k, device="cuda", generator=g) * 0.05
    return X.bfloat16(), W.bfloat16()


def values(q, s):
    s = s.double().repeat_interleave(128, 1)[:, :q.shape[1]]
    return q.double() * (s if s.shape[0] == q.shape[0] else s.repeat_interleave(128, 0)[:q.shape[0]])


def check(got, q, s, w8):
    A, B = values(q, s), values(w8.q, w8.scale)
    want, S = A @ B.t(), A.abs() @ B.abs().t()
    bound = (128 + -(-q.shape[1] // 128) + 4 + 8) * 2.0 ** -23 * S
    err = (got.double() - want).abs()
    assert (err <= bound + torch.finfo(got.dtype).eps / 2 * (want.abs() + bound)).all()


# with the advertised workspace alone, the parts' sums of the first three once lay over X
@pytest.mark.parametrize("m,n,k", [(2560, 1024, 20000), (2048, 1536, 28672), (1715, 1344, 16384), (1537, 1701, 20000),
                                   (200, 19712, 16384)])
def test_frozen_head_with_a_long_contraction(m, n, k):
    assert lce.fp8_matmul_workspace_size(m, n, k) > 1024   # in parts
    X, W = make(m, n, k)
    w8 = lce.fp8_weight(W, transpose=False)
    q, s = lce.quantize_fp8(X)
    with torch.no_grad():
        got = lce.fp8_linear(X, w8)
        check(got, q, s, w8)
        assert torch.equal(got, lce.fp8_matmul(q, s, w8.q, w8.scale))
        assert torch.equal(got, lce.fp8_linear(X, W))


@pytest.mark.parametrize("m,n,k", [(2560, 1024, 20000), (200, 19712, 16384)])
def test_workspaces_of_any_size(m, n, k):
    # the advertised bytes, a little more, as many as parts take, and a large one; nothing beside it is written
    X, W = make(m, n, k)
    w8 = lce.fp8_weight(W, transpose=False)
    q, s = lce.quantize_fp8(X)
    L, need = lce.lib(), ctypes.c_size_t(0)
    assert L.lce_fp8_linear_workspace_size(m, k, ctypes.byref(need)) == 0
    need = need.value
    parts = lce.fp8_matmul_workspace_size(m, n, k) - 1024
    assert parts > 0
    full = -(-need // 1024) * 1024 + parts
    whole = lce.fp8_matmul(q, s, w8.q, w8.scale, ws=torch.empty(1024, dtype=torch.uint8, device="cuda"))
    shared = lce.fp8_matmul(q, s, w8.q, w8.scale)
    for size, want in ((need, whole), (need + 4096, whole), (full - 1, whole), (full, shared), (full + (64 << 20), shared)):
        guard = torch.full((size + 4096,), 85, dtype=torch.uint8, device="cuda")
        ws = guard[2048:2048 + size]
        out = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
        st = L.lce_fp8_linear(X.data_ptr(), 0, k, w8.q.data_ptr(), w8.q.stride(0), w8.scale.data_ptr(),
                              *w8.scale.stride(), m, n, k, out.data_ptr(), n, 0, ws.data_ptr(), size,
                              torch.cuda.current_stream().cuda_stream)
        assert st == 0 and lce.read_status(ws) == 0
        assert torch.equal(out, want), size
        assert (guard[:2048] == 85).all() and (guard[2048 + size:] == 85).all()
    check(whole, q, s, w8)
    check(shared, q, s, w8)


def test_in_parts_captured_and_with_a_gradient():
    m, n, k = 2560, 1024, 20000
    X, W = make(m, n, k)
    w8 = lce.fp8_weight(W)
    with torch.no_grad():
        want = lce.fp8_linear(X, w8)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = lce.fp8_linear(X, w8)
    for _ in range(3):
        got.zero_()
        graph.replay()
        assert torch.equal(got, want)
    Xg = X.clone().requires_grad_()
    Z = lce.fp8_linear(Xg, w8)
    assert torch.equal(Z, want)
    dZ = torch.randn(m, n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).bfloat16()
    (dX,) = torch.autograd.grad(Z, Xg, dZ)
    q, s = lce.quantize_fp8(dZ)
    assert torch.equal(dX, lce.fp8_matmul(q, s, w8.q_t, w8.scale_t))
    side = torch.cuda.Stream()                 # two at once, each with a workspace of its own
    side.wait_stream(torch.cuda.current_stream())
    with torch.no_grad():
        for _ in range(4):
            with torch.cuda.stream(side):
                a = lce.fp8_linear(X, w8)
            b = lce.fp8_linear(X, w8)
            torch.cuda.synchronize()
            assert torch.equal(a, want) and torch.equal(b, want)
