"""4-bit products against bounds that a lost group of weights would break, and where they have to be exact."""
import math

import numpy as np
import pytest
import torch

import linear_cross_entropy_chunked_gb300 as lce
from tests.test_gpu_int4 import HALF, values, weight

pytestmark = pytest.mark.gpu

SHAPES = [(1, 16, 128), (2, 17, 31), (1, 300, 1600), (1, 129, 14000), (2, 200, 8200), (4, 70, 4096), (6, 65, 777),
          (8, 300, 1600), (9, 200, 1000), (33, 130, 8200), (7, 140, 14000), (64, 257, 512), (97, 130, 1601), (200, 300, 8192)]


def bound_of(x, W, group, dtype):
    """Per result, from the sum of the products' magnitudes A. A product of 16 k adds 17 terms on a grid that is cut, not
    rounded, at 2^-23 of the largest: group / 16 of them follow one another. The groups' sums go through two
    roundings each (the scale's product, the addition; a product of more warps than one adds 16 parts), in an order that
    may put any group first. bf16 tokens are rounded to 2^-39 of their largest magnitude where they are below 2^-29 of
    it. One rounding to the type."""
    A = np.abs(x) @ np.abs(W).T
    steps = 17 * max(1, group // 16) * 2.0 ** -23 + 2 * (math.ceil(x.shape[1] / group) + 32) * 2.0 ** -24
    small = 2.0 ** -40 * np.abs(x).max(1)[:, None] * np.abs(W).sum(1)[None] if dtype == torch.bfloat16 else 0.0
    most = steps * A + small
    return most + HALF[dtype] * (np.abs(x @ W.T) + most) + 2.0 ** -25


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("m,v,d", SHAPES)
def test_no_group_is_lost(m, v, d, group, dtype):
    g = torch.Generator().manual_seed(m + d)
    X = torch.randn(m, d, generator=g).to(dtype)
    w = weight(v, d, group, dtype, m + v)
    W, x = values(w, d), X.double().numpy()
    bound = bound_of(x, W, group, dtype)
    for k in range(0, d, group):   # (the bound would tell if any one were)
        assert (np.abs(x[:, k:k + group] @ W[:, k:k + group].T) > 2 * bound).mean() > 0.25
    Z = lce.int4_linear(X.cuda(), w).double().cpu().numpy()
    assert (np.abs(Z - x @ W.T) <= bound).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("m,v,d", SHAPES)
def test_sums_that_are_exact(m, v, d, group, dtype):
    # whole tokens of -2 .. 2 and scales of 1 and 1/2: every sum is a multiple of 1/2 below 2^18, exact in fp32 in any
    # order, so that the result is the exact one, rounded once
    g = torch.Generator().manual_seed(m * d)
    X = torch.randint(-2, 3, (m, d), generator=g).to(dtype)
    q = weight(v, d, group, dtype, v)
    scale = (torch.randint(1, 3, q.scale.shape, generator=g).double() / 2).to(dtype).cuda()
    scale[:, ::5] *= -1            # (a checkpoint's scales may be negative)
    w = lce.Int4Weight(q.q, scale, group)
    want = torch.from_numpy(X.double().numpy() @ values(w, d).T)
    # fp16 ends at 65504
    if dtype == torch.float16:
        assert want.abs().max() < 65504
    assert torch.equal(lce.int4_linear(X.cuda(), w).cpu(), want.to(dtype))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("m", [1, 2, 40])
def test_every_weight_by_itself(m, group, dtype):
    # tokens that are 1 at one place and 0 elsewhere give a column of the weight, rounded once: all places of an odd
    # row for a batch; for one and two tokens those about the ends of groups, units and chunks
    d, v = 3001, 37
    w = weight(v, d, group, dtype, m)
    want = torch.from_numpy(values(w, d)).to(dtype)
    places = range(d) if m == 40 else sorted({p + o for p in range(0, d + 64, 32 if m == 1 else 128) for o in (-1, 0, 1)}
                                             & set(range(d)))
    places = list(places)
    for at in range(0, len(places), m):
        some = (places[at:at + m] * m)[:m]
        X = torch.zeros(m, d, dtype=dtype)
        X[torch.arange(m), torch.tensor(some)] = 1
        assert torch.equal(lce.int4_linear(X.cuda(), w).cpu(), want[:, some].T)
