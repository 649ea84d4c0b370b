"""Tokens far below the largest: where the borders of the cumulative distribution lie.

A weight is a whole number of units of 2^-43 of the largest, rounded to nearest: each is off by at most half
a unit, 0.29 units in the mean square where the logits differ. So the weight up to token i is off by at most
6 * 0.29 sqrt(i) units (six standard deviations of i independent roundings) or, for equal logits, by i / 2, and
the share C_i of it in the total S by that plus C_i times the same for all V; the exponential adds 2^-30 of C_i. A
cut in place of the rounding would be off by i / 2 units for logits that differ too."""
import numpy as np
import pytest
import torch

import linear_cross_entropy_chunked_gb300 as lce
from oracle import ops_oracle

pytestmark = pytest.mark.gpu

UNIT = 2.0 ** -43


def borders(z):
    w = np.exp(z.astype(np.longdouble) - z.max())
    c = np.cumsum(w)
    return c / c[-1], float(c[-1])


def check(z, dtype, draws, bound, **settings):
    """z: the tail first, the one likely token last. `bound`: units by which the first i weights are off."""
    Z = torch.from_numpy(z).to(dtype)
    c, S = borders(Z.double().numpy())
    share = float(c[-2])                       # of the whole tail
    u = (share * (np.arange(draws) + 0.5) / draws).astype(np.float32)
    tokens, logprobs = lce.sample_logits(Z.cuda().expand(draws, -1).contiguous(), torch.from_numpy(u).cuda(), **settings)
    t = tokens.cpu().numpy()
    assert (t < len(z) - 1).all()
    V = len(z)
    before = np.where(t > 0, c[np.maximum(t - 1, 0)], 0).astype(np.float64)
    upto, u = c[t].astype(np.float64), u.astype(np.float64)

    def off(i, share):
        return (bound(i) + share * bound(V)) * UNIT / S + 2.0 ** -30 * share
    assert (u >= before - off(t, before)).all(), ((before - u) / off(t, before)).max()
    assert (u < upto + off(t + 1, upto)).all(), ((u - upto) / off(t + 1, upto)).max()
    want = Z.double().numpy()[t] - Z.double().max().item() - np.log(S)
    assert (np.abs(logprobs.cpu().double().numpy() - want) <= 2.0 ** -22 * (np.abs(want) + 1)).all()


def independent(i):
    return 6 * 0.29 * np.sqrt(i) + 1


def equal(i):
    return 0.5 * i + 1


@pytest.mark.parametrize("v", [32000, 128256, 262144, 1 << 20])
@pytest.mark.parametrize("gap", [16.0, 22.0, 27.0])
def test_a_long_tail_of_different_logits(v, gap):
    z = (np.random.default_rng(v).standard_normal(v) * 0.5).astype(np.float32)
    z[-1] = gap
    check(z, torch.float32, 64, independent)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("gap", [16.0, 24.75, 26.0, 27.0])
def test_a_long_tail_of_equal_logits(gap, dtype):
    # (2^43 exp(-gap) is 0.87, 0.86, 0.94 and 0.53 above a whole number: a cut would be off by that much per token)
    z = np.zeros(128256, np.float32)
    z[-1] = gap
    check(z, dtype, 64, equal)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_far_logits_have_no_weight(dtype):
    # beyond exp(-x) = 2^-44 a token is never drawn, however far: distances over temperatures from just beyond it
    # to the ends of the types, infinities and NaN among them
    lowest = torch.finfo(dtype).min
    n, v = 64, 4096
    g = torch.Generator().manual_seed(5)
    for t in (1.0, 1e-4, 3e-5, 1e-3):
        far = torch.cat([-31.0 * t - 10 ** (torch.rand(v - 4, generator=g) * 9 - 3), torch.tensor([-float("inf"), float("nan"), lowest])])
        z = torch.cat([torch.zeros(1), far.clamp(min=lowest)]).to(dtype)
        z[1:] = torch.where(z[1:] > -31.5 * t, torch.tensor(-float("inf"), dtype=dtype), z[1:])
        u = torch.cat([1 - torch.rand(n - 2, generator=g) * 2.0 ** -20, torch.tensor([0.0, 1 - 2.0 ** -24])]).float()
        u = u.clamp(max=1 - 2.0 ** -24)
        tokens, logprobs = lce.sample_logits(z.cuda().expand(n, -1).contiguous(), u.cuda(), temperature=t)
        assert (tokens == 0).all() and (logprobs == 0).all(), t
        z = z.flip(0)                          # the one token last: a weight before it would be drawn at u = 0
        tokens, logprobs = lce.sample_logits(z.cuda().expand(n, -1).contiguous(), (u * 0).cuda(), temperature=t)
        assert (tokens == v - 1).all() and (logprobs == 0).all(), t


@pytest.mark.parametrize("settings", [{}, {"top_p": 0.5}, {"top_k": 700}, {"min_p": 0.5}])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_ends_of_the_temperature(dtype, settings):
    # an infinite one makes all finite logits equally likely (the first by index are kept), a huge one nearly so;
    # masked logits stay out, and a tiny one leaves the largest logit alone
    n, v = 9, 3000
    g = torch.Generator().manual_seed(7)
    z = (torch.randn(n, v, generator=g) * 3).to(dtype)
    z[:, ::5] = -float("inf")
    z[:, 3::5] = float("nan")
    t = torch.tensor([float("inf"), 1e38, 1e30, 3e-39, 1e-37, 1e-30, 1.0, 1e5, 3.4e38])
    u = torch.rand(n, generator=g)
    ref = ops_oracle.sample(z.double().numpy(), u.double().numpy(), t.double().numpy(), **settings)
    tokens, logprobs = lce.sample_logits(z.cuda(), u.cuda(), temperature=t.cuda(), **settings)
    np.testing.assert_array_equal(tokens.cpu().numpy(), ref["tokens"])
    err = np.abs(logprobs.cpu().double().numpy() - ref["logprobs"])
    assert (err <= 2.0 ** -22 * (ref["x"] + ref["ls"] + 1)).all()
