"""Losses on answers over logits that are masked with finite numbers of any size, and at temperatures down to the
smallest one, against the fp64 oracle."""
import math

import numpy as np
import pytest
import torch

import linear_cross_entropy_chunked_gb300 as lce
from oracle import answers_oracle as ao
from tests.test_gpu_policy import HALF, TINY, check_gradients, cpu64, rows_like, with_coefs

pytestmark = pytest.mark.gpu

MASKS = [-1e9, -1e10, -1e20, -1e30, -1e38]
STEP = 2.0 ** -24


def row_bound(Z, y, temperature):
    """Per row, how far an fp32 log probability may be off. A term exp(x), x = (z - max) / T, moves by its exponent's
    roundings: the distance, log2(e) / T (three: 1 / T, log2(e), their product) and the product, five half steps of
    |x|. Beyond 110 a term, whatever the roundings, is below e^-109, nothing beside the sum of 1 or more. ex2 is off by
    2^-22, the sum goes through 40 + log2 v additions, and each of them and of the maxima in between through one
    exponential more. The label's own distance is rounded three times, and the result once."""
    v = Z.shape[1]
    ok = (y >= 0) & (y < v)
    x = (Z - Z.max(1, keepdims=True)) / temperature
    far = np.minimum(-x.min(1), 110.0)
    label = np.where(ok, -x[np.arange(len(y)), np.where(ok, y, 0)], 0.0)
    return (2 * 5 * far + 4 * label + 2 * (2 + 40 + math.log2(v + 1)) + 8 + 2 * math.log(v + 1)) * STEP


def check_policy(Z, y, got, o, temperature, dtype):
    loss, logprobs, dZ = got
    lb = row_bound(cpu64(Z), y, temperature)
    assert (np.abs(cpu64(logprobs) - o["logprobs"]) <= np.where(o["ok"], lb, 0.0)).all()
    rel = 2 * lb + 12 * STEP
    n = max(1, o["ok"].sum())
    assert abs(loss.item() - o["loss"]) <= (rel * o["terms"]).sum() / n + 2.0 ** -23 * abs(o["loss"])
    if dZ is None:
        return
    onehot = np.zeros_like(o["p"])
    onehot[np.flatnonzero(o["ok"]), y[o["ok"]]] = 1.0
    # (an exponential below fp32's smallest normal number is 0: up to 2^-126 of the coefficient, which is 1 / T and
    # more, is missing; twice that with the roundings around it)
    rounding = HALF[dtype] * np.abs(o["dZ"]) + 2 * TINY[dtype] + 2.0 ** -125 * o["mass"][:, None]
    bound = (2 * rel * o["mass"])[:, None] * (o["p"] + onehot) + rounding
    assert (np.abs(cpu64(dZ) - o["dZ"]) <= bound).all()


def check_preference(Z, y, off, got, o, beta, dtype):
    loss, seq, dZ = got
    lb = np.where(o["ok"], row_bound(cpu64(Z), y, 1.0), 0.0)
    sb = np.array([lb[a:b].sum() for a, b in zip(off, off[1:])]) + 2.0 ** -22 * np.abs(o["seq_logprobs"])
    assert (np.abs(cpu64(seq) - o["seq_logprobs"]) <= sb).all()
    P = len(sb) // 2
    m = beta * (sb[:P] + sb[P:]) + 2.0 ** -22 * np.abs(o["margin"])
    assert abs(loss.item() - o["loss"]) <= m.max() + 2.0 ** -21 * (1 + abs(o["loss"]))
    if dZ is None:
        return
    onehot = np.zeros_like(o["p"])
    onehot[np.flatnonzero(o["ok"]), y[o["ok"]]] = 1.0
    # the slope's sigmoid moves by less than its margin (relative to the smaller one of the two: e^m)
    rel = (np.expm1(m.max()) + 2 * lb + 2.0 ** -19)[:, None]
    bound = rel * np.abs(o["coef"])[:, None] * (o["p"] + onehot) + HALF[dtype] * np.abs(o["dZ"]) + 2 * TINY[dtype] + 1e-37
    assert (np.abs(cpu64(dZ) - o["dZ"]) <= bound).all()


def masked(v, mask, seed):
    """Eight rows: most of a row masked, all but the label, runs that a thread or a whole CTA sees nothing beside, the
    head and the tail, the whole row; and one whose largest logits are -mask. Labels are not masked."""
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(8, v, generator=g) * 3
    y = torch.randint(0, v, (8,), generator=g)
    keep = [torch.zeros(v, dtype=torch.bool) for _ in range(8)]
    keep[0] = torch.rand(v, generator=g) < 0.03
    keep[2][: v // 2] = True
    keep[3][v // 2:] = True
    keep[4] = (torch.arange(v) // 8) % 3 != 1        # a thread's vectors of 8 (or two of 4), here and there
    keep[5] = torch.arange(v) >= 5
    for r in range(6):
        keep[r][y[r]] = True
        z[r][~keep[r]] = mask
    z[6] = mask
    z[7][y[7]] = -mask
    z[7][v // 3] = -mask
    return z, y


def policy_inputs(Z, y, temperature, seed):
    n = len(y)
    g = torch.Generator().manual_seed(seed)
    logp = torch.from_numpy(ao.log_softmax_of(cpu64(Z), y.numpy(), temperature)[0])
    moved = 0.2 * torch.randn(n, generator=g)
    for border in (0.8, 1.2):   # (no ratio so near to a border that fp32 could not say on which side)
        moved = torch.where((torch.exp(-moved) - border).abs() < 0.01, moved + 0.03, moved)
    return (torch.randn(n, generator=g), (logp + moved).float(),
            (logp + 0.2 * torch.randn(n, generator=g)).float())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("v,layout", [(17, "dense"), (33, "odd"), (777, "odd"), (5003, "dense"), (50257, "dense"),
                                      (128256, "padded"), (600001, "odd")])
def test_finite_masks(v, layout, mask, dtype):
    z, y = masked(v, mask, v)
    Z = rows_like(z, layout, dtype)
    a, old, ref = policy_inputs(Z, y, 1.0, 1)
    args = [t.cuda() for t in (y, a, old, ref)]
    o = ao.policy(cpu64(Z), y.numpy(), a.numpy(), old.numpy(), ref.numpy(), beta=0.04)
    for grad in (True, False):
        check_policy(Z, y.numpy(), lce.policy_logits(Z, *args, beta=0.04, grad=grad), o, 1.0, dtype)
    off = np.array([0, 2, 4, 6, 8])
    seq = ao.preference(cpu64(Z), y.numpy(), off)["seq_logprobs"]
    ref = torch.from_numpy(seq + [0.3, -0.2, 0.1, 0.4]).float()
    o = ao.preference(cpu64(Z), y.numpy(), off, ref.numpy(), 0.5)
    for grad in (True, False):
        got = lce.preference_logits(Z, y.cuda(), torch.from_numpy(off).cuda(), ref.cuda(), beta=0.5, grad=grad)
        check_preference(Z, y.numpy(), off, got, o, 0.5, dtype)


@pytest.mark.parametrize("temperature", [0.1, 1e-2, 1e-3, 1e-6, 1e-9, 2.0 ** -64, 30.0, 1e9])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=str)
@pytest.mark.parametrize("v,layout", [(9, "odd"), (1000, "dense"), (50257, "dense"), (600001, "odd")])
def test_temperatures(v, layout, dtype, temperature):
    if dtype == torch.float16 and temperature < 1e-3:
        temperature = 1e-3      # (a gradient is 1 / T: fp16 has none of them below)
    n = 6
    g = torch.Generator().manual_seed(v)
    z = torch.randn(n, v, generator=g) * 4
    if dtype == torch.float16:
        z[1, 1:] = -6e4         # a mask of this type
    Z = rows_like(z, layout, dtype)
    y = Z.float().argmax(1).cpu()        # the most likely token: log p is 0, or that of a tie
    y[5] = int(torch.randint(0, v, (1,), generator=g))
    a, old, ref = policy_inputs(Z, y, temperature, 2)
    a[5] = 0.0                           # (an unlikely token's log probability is checked alone)
    args = [t.cuda() for t in (y, a, old)]
    exact = old.double().numpy()
    exact[5] = ao.log_softmax_of(cpu64(Z), y.numpy(), temperature)[0][5]
    o = ao.policy(cpu64(Z), y.numpy(), a.numpy(), exact, temperature=temperature)
    for grad in (True, False):
        got = lce.policy_logits(Z, *args, temperature=temperature, grad=grad)
        check_policy(Z, y.numpy(), got, o, temperature, dtype)
    assert torch.isfinite(got[1]).all()


@pytest.mark.parametrize("temperature", [0.05, 1e-3, 1e-4, 1e-5, 1e-6, 1e-9, 2.0 ** -64, 1e9])
@pytest.mark.parametrize("n,v,chunk", [(7, 129, 1024), (300, 1000, 1024), (400, 5003, 64)])
def test_temperatures_over_the_head(n, v, chunk, temperature):
    # values of a quarter to three: every product and sum of a logit is exact, in whichever order it is formed, so
    # that nothing but the softmax is looked at
    d = 64
    g = torch.Generator().manual_seed(n + v)
    H = (torch.randint(-12, 13, (n, d), generator=g) / 4).bfloat16()
    W = (torch.randint(-12, 13, (v, d), generator=g) / 4).bfloat16()
    Z = (H.double() @ W.double().t()).numpy()
    y = torch.from_numpy(Z.argmax(1))    # the most likely token: log p is 0, or that of a tie
    y[torch.rand(n, generator=g) < 0.3] = -100
    y[0] = 3                             # an unlikely one, whose log probability is checked alone
    a, old, ref = policy_inputs(torch.from_numpy(Z), y, temperature, 2)
    a[0] = 0.0
    args = [t.cuda() for t in (H, W, y, a, old)]
    how = dict(temperature=temperature, chunk=chunk)
    exact = old.double().numpy()
    exact[0] = ao.log_softmax_of(Z, y.numpy(), temperature)[0][0]
    o = ao.policy(Z, y.numpy(), a.numpy(), exact, temperature=temperature)
    loss, logprobs, dH, dW = lce.policy_fwd_bwd(*args, **how)
    lb = row_bound(Z, y.numpy(), temperature)
    assert (np.abs(cpu64(logprobs) - o["logprobs"]) <= np.where(o["ok"], lb, 0.0)).all()
    lb = lb[1:].max()
    count = o["ok"].sum()
    assert abs(loss.item() - o["loss"]) <= (2 * lb + 2.0 ** -20) * o["terms"].sum() / count
    check_gradients(dH, dW, H, W, with_coefs(o, y, o["mass"]), lb)
    frozen = lce.policy_fwd_bwd(*args, **how, compute_dW=False)
    assert torch.equal(frozen[0], loss) and torch.equal(frozen[1], logprobs)
    check_gradients(frozen[2], None, H, W, with_coefs(o, y, o["mass"]), lb)
    l2, lp2 = lce.policy_forward(*args, **how)
    assert torch.equal(lp2, logprobs) and torch.equal(l2, loss)
