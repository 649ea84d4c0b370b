"""Gradient norm and clipping against the fp64 oracle.

The norm: a thread sums at most 32 products in two fp32 chains of 16 fused steps (each rounding
at most 2^-24 of the sum so far: 16 * 2^-24, plus one for their sum), the rest is held in pairs
and fp64; its root halves that, and is rounded once: within 10 * 2^-24 relative (norm 1, with
no root: 19 * 2^-24). The factor adds three roundings, the product one of its own type."""
import math

import numpy as np
import pytest
import torch

import linear_cross_entropy_chunked_gb300 as lce
from oracle import ops_oracle

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
NORM_REL = 19 * 2.0 ** -24
FACTOR_REL = NORM_REL + 3 * 2.0 ** -24


def make(sizes, dtype, seed, scale=1.0, offset=0):
    g = torch.Generator().manual_seed(seed)
    kinds = [dtype] * len(sizes) if dtype in DTYPES else [list(DTYPES)[i % 3] for i in range(len(sizes))]
    host = [(torch.randn(n, generator=g) * scale * 10 ** float(torch.rand((), generator=g))).to(DTYPES[k])
            for n, k in zip(sizes, kinds)]
    return host, [torch.cat([torch.zeros(offset, dtype=h.dtype), h]).cuda()[offset:] for h in host]


def check(host, dev, max_norm, norm_type=2.0, out=None):
    norm = lce.clip_grad_norm(dev, max_norm, norm_type=norm_type, out=out)
    want, scaled = ops_oracle.clip([h.double().numpy() for h in host], max_norm, norm_type)
    assert norm.dtype == torch.float32 and norm.shape == ()
    assert abs(norm.item() - want) <= NORM_REL * want
    for h, w, d in zip(host, scaled, dev if out is None else out):
        half = torch.finfo(h.dtype).eps / 2
        tiny = float(torch.finfo(h.dtype).smallest_normal) * torch.finfo(h.dtype).eps   # subnormal step
        err = np.abs(d.double().cpu().numpy() - w)
        assert (err <= (half + FACTOR_REL) * np.abs(w) + tiny / 2).all()
    return norm


@pytest.mark.parametrize("norm_type", [2.0, 1.0, math.inf])
@pytest.mark.parametrize("dtype", list(DTYPES) + ["mixed"])
@pytest.mark.parametrize("sizes", [[1], [3], [7, 1, 9], [0, 5, 0], [8, 16, 24], [1000, 1, 4097, 33],
                                   [8191], [16384], [16385, 3, 40000], [1_000_003]])
def test_clip_in_place(sizes, dtype, norm_type):
    host, dev = make(sizes, dtype, sum(sizes) + len(sizes))
    norm = ops_oracle.grad_norm([h.double().numpy() for h in host], norm_type)
    check(host, dev, 0.3 * norm, norm_type)


@pytest.mark.parametrize("n", [63, 64, 65, 1024, 1025, 2500])
def test_many_tensors(n):
    g = torch.Generator().manual_seed(n)
    host, dev = make([int(k) for k in torch.randint(0, 300, (n,), generator=g)], "mixed", n)
    check(host, dev, 5.0)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("offset", [1, 2, 3, 5])
def test_alignment(dtype, offset):
    sizes = [5, 100, 20011]
    host, dev = make(sizes, dtype, offset, offset=offset)
    out = [torch.full_like(d, 7.0) for d in dev]
    check(host, dev, 1.0, out=out)
    for h, d in zip(host, dev):
        assert torch.equal(h, d.cpu())   # not in place
    shifted = [torch.full((d.numel() + 2,), 7.0, dtype=d.dtype, device="cuda") for d in dev]
    check(host, dev, 1.0, out=[s[1:-1] for s in shifted])
    for s in shifted:
        assert s[0] == 7 and s[-1] == 7  # nothing beside the tensor is written
    check(host, dev, 1.0)


def test_neighbours_are_left_as_they_were():
    flat = torch.randn(1 << 16, device="cuda").bfloat16()
    host = flat.cpu()
    parts = [flat[3:1001], flat[1001:1002], flat[2000:40001]]
    check([p.cpu() for p in parts], parts, 0.1)
    keep = torch.ones(1 << 16, dtype=torch.bool)
    keep[3:1002] = False
    keep[2000:40001] = False
    assert torch.equal(flat.cpu()[keep], host[keep])


def test_layouts():
    g = torch.randn(64, 48, 5, device="cuda").permute(2, 0, 1)
    host = g.cpu().clone()
    check([host], [g], 1.0)
    out = torch.empty_like(g)
    g.copy_(host)
    check([host], [g], 1.0, out=[out])
    with pytest.raises(ValueError):
        lce.clip_grad_norm(torch.randn(8, 8, device="cuda")[:, :4], 1.0)


def test_below_the_limit_nothing_is_written():
    host, dev = make([1000, 70001], "mixed", 5)
    before = [d.clone() for d in dev]
    check(host, dev, 1e9)
    assert all(torch.equal(a, b) for a, b in zip(before, dev))
    out = [torch.zeros_like(d) for d in dev]
    check(host, dev, 1e9, out=out)
    assert all(torch.equal(a, b) for a, b in zip(before, out))


def test_special_values():
    for kind in (2.0, 1.0, math.inf):
        g = torch.ones(5000, device="cuda")
        g[4321] = math.nan
        assert math.isnan(lce.clip_grad_norm(g, 1.0, norm_type=kind).item())
        assert torch.isnan(g).all()
        g = torch.ones(5000, device="cuda")
        g[17] = -math.inf
        assert lce.clip_grad_norm(g, 1.0, norm_type=kind).item() == math.inf
        assert (g[:17] == 0).all() and torch.isnan(g[17])
        g = torch.zeros(5000, device="cuda")
        assert lce.clip_grad_norm(g, 1.0, norm_type=kind).item() == 0.0
        g = torch.ones(5000, device="cuda")
        lce.clip_grad_norm(g, 0.0, norm_type=kind)
        assert (g == 0).all()
        g = torch.ones(300, device="cuda", dtype=torch.bfloat16)
        lce.clip_grad_norm(g, math.inf, norm_type=kind)
        assert (g == 1).all()


def test_long_sum():
    # 2^28 equal values: a plain fp32 running sum would stop growing
    g = torch.full((1 << 28,), 0.01, device="cuda")
    want = float(np.float32(0.01)) * 2.0 ** 14
    assert abs(lce.grad_norm(g).item() - want) <= NORM_REL * want
    want = float(np.float32(0.01)) * 2.0 ** 28
    assert abs(lce.grad_norm(g, norm_type=1).item() - want) <= NORM_REL * want


def test_norm_alone_matches_and_repeats():
    host, dev = make([300_007, 11, 5000], "mixed", 8)
    before = [d.clone() for d in dev]
    runs = [lce.grad_norm(dev).item() for _ in range(3)]
    assert len(set(runs)) == 1
    assert all(torch.equal(a, b) for a, b in zip(before, dev))
    assert lce.clip_grad_norm(dev, 1.0).item() == runs[0]


def test_graphs_and_stream():
    host, dev = make([4000, 9000], "fp32", 9)
    ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    outs = [[torch.empty_like(d) for d in dev] for _ in range(2)]
    norms, graphs = [], []
    for out, m in zip(outs, (1.0, 3.0)):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            norms.append(lce.clip_grad_norm(dev, m, out=out, ws=ws))   # both use one workspace
        graphs.append(graph)
    for seed in (10, 11):
        host, new = make([4000, 9000], "fp32", seed)
        for d, x in zip(dev, new):
            d.copy_(x)
        for graph, norm, out, m in zip(graphs, norms, outs, (1.0, 3.0)):
            graph.replay()
            want, scaled = ops_oracle.clip([h.double().numpy() for h in host], m)
            assert abs(norm.item() - want) <= NORM_REL * want
            for o, w in zip(out, scaled):
                assert (np.abs(o.double().cpu().numpy() - w) <= (2.0 ** -24 + FACTOR_REL) * np.abs(w)).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    norm = lce.clip_grad_norm(dev, 1.0, out=outs[0], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert abs(norm.item() - want) <= NORM_REL * want
