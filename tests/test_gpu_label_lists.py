"""The weight gradient of losses on answers where a chunk has so many rows that its labels' lists are found pass by pass."""
import numpy as np
import pytest
import torch

import linear_cross_entropy_chunked_gb300 as lce
from oracle import answers_oracle as ao
from tests.test_gpu_policy import check_gradients, cpu64, logp_bound, with_coefs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ignored", [0.0, 0.4])
@pytest.mark.parametrize("n,v", [(16384, 50), (16385, 50), (16385, 3), (16500, 3001), (40001, 503)])
def test_many_rows_in_one_chunk(n, v, ignored):
    # below and above the number of rows from which it is so; labels that thousands of rows have, that some eight have, that one
    # has; the remainders of up to eight rows are added to a label's row of dW, without which frequent or rare
    # labels' rows would be off by more than the bound
    d = 16
    g = torch.Generator().manual_seed(n + v)
    H = torch.randn(n, d, generator=g).bfloat16()
    W = (torch.randn(v, d, generator=g) / 2).bfloat16()
    y = torch.randint(0, v, (n,), generator=g)
    y[n // 2:n // 2 + 50] = v - 1
    y[torch.rand(n, generator=g) < ignored] = -100
    a = torch.randn(n, generator=g)
    loss, logprobs, dH, dW = lce.policy_fwd_bwd(H.cuda(), W.cuda(), y.cuda(), a.cuda(), chunk=n)
    Z = (H.double() @ W.double().t()).numpy()
    o = ao.policy(Z, y.numpy(), a.numpy())
    lb = logp_bound(Z, 1.0, v) + 2 * (2 * d + 8) * 2.0 ** -24 * float((H.double().abs() @ W.double().abs().t()).max())
    assert np.abs(cpu64(logprobs) - o["logprobs"]).max() <= lb
    check_gradients(dH, dW, H, W, with_coefs(o, y, o["mass"]), lb)
    again = lce.policy_fwd_bwd(H.cuda(), W.cuda(), y.cuda(), a.cuda(), chunk=n)
    assert all(torch.equal(p, q) for p, q in zip(again, (loss, logprobs, dH, dW)))


@pytest.mark.parametrize("v", [3, 2003, 30000])
def test_both_ways_give_the_same(v):
    # one row more, which does not count: the rows that do are the same, their lists are found in the other way, and nothing
    # else of dW changes
    n, d = 16384, 16
    g = torch.Generator().manual_seed(v)
    H = torch.randn(n + 1, d, generator=g).bfloat16().cuda()
    W = (torch.randn(v, d, generator=g) / 2).bfloat16().cuda()
    y = torch.randint(0, v, (n + 1,), generator=g)
    y[torch.rand(n + 1, generator=g) < 0.2] = -100
    y[n] = -100
    y, a = y.cuda(), torch.randn(n + 1, generator=g).cuda()
    one = lce.policy_fwd_bwd(H, W, y, a, chunk=n + 1)
    two = lce.policy_fwd_bwd(H[:n], W, y[:n], a[:n], chunk=n + 1)
    assert torch.equal(one[3], two[3]) and torch.equal(one[1][:n], two[1])
