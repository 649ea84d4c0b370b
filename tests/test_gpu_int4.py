"""The 4-bit linear layer against the fp64 oracle."""
import math

import numpy as np
import pytest
import torch

import linear_cross_entropy_chunked_gb300 as lce
from oracle import answers_oracle as ao

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def weight(v, d, group, dtype, seed):
    """Packed values with anything behind the last one of a row, and scales."""
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(0, 256, (v, -(-d // 32) * 16), generator=g, dtype=torch.uint8)
    scale = ((torch.rand(v, -(-d // group), generator=g) + 0.5) * 0.01).to(dtype)
    return lce.Int4Weight(q.cuda()[:, :(d + 1) // 2], scale.cuda(), group)


def values(w, d):
    return ao.int4_values(w.q.cpu().numpy(), w.scale.double().cpu().numpy(), w.group, d)


def check(Z, X, W):
    """Sums of d products: at most d / 4 + 64 roundings (to nearest or cut) of the magnitudes that are
    summed; and one rounding to the type."""
    x = X.double().cpu().numpy()
    want = x @ W.T
    d = x.shape[1]
    most = np.abs(x) @ np.broadcast_to(np.abs(W).max(1)[:, None], W.shape).T * 8
    bound = (d / 4 + 64) * 2.0 ** -23 * most + HALF[X.dtype] * np.abs(want) + 2.0 ** -25
    err = np.abs(Z.double().cpu().numpy() - want)
    assert (err <= bound).all(), float((err / bound).max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("m,v,d", [(1, 1, 1), (1, 16, 128), (2, 17, 31), (3, 50, 33), (1, 1000, 4096), (8, 300, 1600), (5, 129, 777),
                                   (9, 200, 1000), (16, 64, 2048), (17, 333, 640), (40, 100, 96), (33, 1003, 8200), (7, 40, 14000),
                                   (64, 257, 512), (129, 130, 1600), (200, 600, 384), (300, 70, 8192)])
def test_against_the_oracle(m, v, d, group, dtype):
    g = torch.Generator().manual_seed(m + d)
    X = (torch.randn(m, d, generator=g) * torch.exp(torch.randn(1, d, generator=g))).to(dtype).cuda()
    w = weight(v, d, group, dtype, m + v)
    Z = lce.int4_linear(X, w)
    assert Z.shape == (m, v) and Z.dtype == dtype
    check(Z, X, values(w, d))
    assert torch.equal(Z, lce.int4_linear(X, w))


@pytest.mark.parametrize("m", [1, 6, 30, 100])
@pytest.mark.parametrize("d", [160, 1001])
def test_strides_and_outputs(m, d):
    v, dtype = 211, torch.bfloat16
    g = torch.Generator().manual_seed(d)
    buf = torch.full((m, d + 5), math.nan, dtype=dtype, device="cuda")
    X = buf[:, 3:3 + d]
    X.copy_(torch.randn(m, d, generator=g))
    w = weight(v, d, 64, dtype, 1)
    wide = torch.zeros(v, 1024, dtype=torch.uint8, device="cuda")
    wide[:, :w.q.shape[1]] = w.q
    scales = torch.full((v, 37), math.nan, dtype=dtype, device="cuda")
    scales[:, 1:1 + w.scale.shape[1]] = w.scale
    w2 = lce.Int4Weight(wide[:, :w.q.shape[1]], scales[:, 1:1 + w.scale.shape[1]], 64)
    out = torch.full((m, v + 9), math.nan, dtype=dtype, device="cuda")
    Z = lce.int4_linear(X, w2, out=out[:, 1:1 + v])
    assert Z.data_ptr() == out[:, 1:].data_ptr()
    check(Z, X, values(w, d))
    assert torch.isnan(out[:, 0]).all() and torch.isnan(out[:, 1 + v:]).all()
    assert torch.equal(Z, lce.int4_linear(X.contiguous(), w))


def test_a_token_does_not_depend_on_the_others():
    # (an infinity or a NaN in one row stays in it; the scale of a bad group reaches its row of the weight only)
    X = torch.randn(12, 300, device="cuda").bfloat16()
    w = weight(100, 300, 32, torch.bfloat16, 3)
    clean = lce.int4_linear(X, w)
    X[4, 7], X[9, 1] = math.nan, math.inf
    Z = lce.int4_linear(X, w)
    keep = [i for i in range(12) if i not in (4, 9)]
    assert torch.equal(Z[keep], clean[keep]) and torch.isnan(Z[4]).all() and not torch.isfinite(Z[9]).any()
    w.scale[50, 2] = math.nan
    Z = lce.int4_linear(X[keep], w)
    assert torch.isnan(Z[:, 50]).all() and torch.isfinite(Z[:, :50]).all() and torch.isfinite(Z[:, 51:]).all()


def test_no_tokens():
    w = weight(10, 64, 32, torch.float16, 1)
    assert lce.int4_linear(torch.empty(0, 64, dtype=torch.float16, device="cuda"), w).shape == (0, 10)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=str)
@pytest.mark.parametrize("v,d,group", [(1, 1, 32), (3, 31, 32), (17, 130, 64), (40, 1000, 128), (5, 4096, 128), (9, 257, 32)])
def test_quantisation(v, d, group, dtype):
    g = torch.Generator().manual_seed(d)
    buf = (torch.randn(v, d + 3, generator=g) * 0.05).to(dtype).cuda()
    W = buf[:, 1:1 + d]
    W[0, :min(d, 40)] = 0
    w = lce.int4_weight(W, group)
    half = dtype if dtype != torch.float32 else torch.bfloat16
    assert w.scale.dtype == half and w.q.shape == (v, (d + 1) // 2)

    def rounded(s):
        return torch.from_numpy(s.astype(np.float32)).to(half).double().numpy()
    x = W.double().cpu().numpy()
    q, s = ao.quantize_int4(x, group, rounded)
    # (a seventh in fp32 is off by 2^-24: a scale next to a tie may be the neighbour)
    got = w.scale.double().cpu().numpy()
    assert (np.abs(got - s) <= 2 * HALF[half] * s).all() and (got != s).mean() <= 0.01
    ratio = x / np.repeat(got, group, 1)[:, :d]
    mine = ao.int4_values(w.q.cpu().numpy(), np.ones_like(got), group, d)
    assert (np.abs(mine - np.clip(ratio, -8, 7)) <= 0.5 + 1e-6).all()
    same = got == s
    near = np.abs(np.abs(ratio - np.floor(ratio)) - 0.5) < 1e-6
    assert ((mine == q) | near | ~np.repeat(same, group, 1)[:, :d]).all()
    W[v // 2, d // 2] = math.inf
    bad = lce.int4_weight(W, group).scale
    assert torch.isnan(bad[v // 2, d // 2 // group]) and torch.isnan(bad).sum() == 1


def test_captured_and_on_a_stream():
    w = weight(3001, 512, 128, torch.bfloat16, 9)
    X = torch.randn(4, 512, device="cuda").bfloat16()
    out = torch.empty(4, 3008, dtype=torch.bfloat16, device="cuda")[:, :3001]
    lce.int4_linear(X, w, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lce.int4_linear(X, w, out=out)
    for _ in range(2):
        X.copy_(torch.randn(4, 512))
        graph.replay()
        assert torch.equal(out, lce.int4_linear(X, w))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    Z = lce.int4_linear(X, w, stream=s)
    s.synchronize()
    assert torch.equal(Z, out)
