"""The preference loss of many pairs, most of them of short or empty answers."""
import numpy as np
import pytest
import torch

import linear_cross_entropy_chunked_gb300 as lce
from oracle import answers_oracle as ao
from tests.test_gpu_policy import HALF, cpu64

pytestmark = pytest.mark.gpu

OFFSETS = 8


def case(pairs, n, v, seed):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(n, v, generator=g) * 2
    y = torch.randint(0, v, (n,), generator=g)
    y[torch.rand(n, generator=g) < 0.2] = -100
    off = torch.cat([torch.tensor([2]), torch.randint(2, n - 1, (2 * pairs - 1,), generator=g).sort().values, torch.tensor([n - 1])])
    return z, y, off, torch.randn(2 * pairs, generator=g)


def expected(z, y, off, ref, beta):
    """(loss of each pair, log probabilities of the sequences, each row's coefficient for a mean), by sums up to each offset."""
    logp, p, ok = ao.log_softmax_of(z, y)
    seq = np.diff(np.concatenate([[0.0], np.cumsum(logp)])[off])
    P = len(seq) // 2
    x = seq - ref
    m = beta * (x[:P] - x[P:])
    slope = -beta * np.exp(-np.logaddexp(0, m)) / P
    sequence = np.searchsorted(off, np.arange(len(y)), side="right") - 1
    inside = (sequence >= 0) & (sequence < 2 * P)
    of = np.where(inside, sequence, 0)
    coef = np.where(inside & ok, np.where(of < P, -slope[of % P], slope[of % P]), 0.0)
    return np.logaddexp(0, -m), seq, coef, p, ok


@pytest.mark.parametrize("pairs,n", [(512, 3000), (513, 3000), (4095, 9000), (4096, 500), (100003, 20000), (1 << 20, 4000)])
def test_many_pairs(pairs, n):
    z, y, off, ref = case(pairs, n, 33, pairs)
    Z = z.cuda()
    loss, seq, dZ = lce.preference_logits(Z, y.cuda(), off.cuda(), ref.cuda(), beta=0.3, reduction="none")
    want, L, coef, p, ok = expected(z.double().numpy(), y.numpy(), off.numpy(), ref.double().numpy(), 0.3)
    # a row's log probability: distances of up to 20, rounded three times, and the sums (fewer than 250 half steps in all)
    rows = np.diff(off.numpy())
    sb = (rows + 1) * 250 * 2.0 ** -24 + 2.0 ** -22 * np.abs(L)
    assert (np.abs(cpu64(seq) - L) <= sb).all()
    mb = 0.3 * (sb[:pairs] + sb[pairs:]) + 2.0 ** -20
    assert (np.abs(cpu64(loss) - want) <= mb).all()
    onehot = np.zeros_like(p)
    onehot[np.flatnonzero(ok), y.numpy()[ok]] = 1.0
    exact = (p - onehot) * coef[:, None] * pairs       # (a loss of each pair has coefficients without the mean's 1 / pairs)
    bound = (4 * mb.max() + 2.0 ** -18) * np.abs(coef[:, None]) * pairs * (p + onehot) + HALF[torch.float32] * np.abs(exact) + 1e-37
    assert (np.abs(cpu64(dZ) - exact) <= bound).all()
    total = lce.preference_logits(Z, y.cuda(), off.cuda(), ref.cuda(), beta=0.3, grad=False)[0]
    assert abs(total.item() - want.mean()) <= mb.mean() + 2.0 ** -22


@pytest.mark.parametrize("pairs", [512, 513, 9000])
def test_offsets_that_do_not_fit_are_taken_as_their_running_maximum(pairs):
    n = 700
    z, y, off, ref = case(pairs, n, 17, pairs)
    bad = off.clone()
    bad[5] = 600
    bad[7] = -3
    bad[pairs + 9] = n + 50
    bad[-2] = 1
    good = bad.clamp(0, n).cummax(0).values
    ws = torch.empty(1 << 21, dtype=torch.uint8, device="cuda")
    args = (z.cuda(), y.cuda())
    a = lce.preference_logits(*args, bad.cuda(), ref.cuda(), ws=ws)
    assert lce.read_status(ws) == OFFSETS and lce.read_status(ws) == 0
    b = lce.preference_logits(*args, good.cuda(), ref.cuda(), ws=ws)
    assert lce.read_status(ws) == 0
    assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("pairs", [512, 600])
def test_over_the_head(pairs):
    n, d, v = 900, 64, 130
    g = torch.Generator().manual_seed(pairs)
    H, W = torch.randn(n, d, generator=g).bfloat16(), (torch.randn(v, d, generator=g) / 4).bfloat16()
    _, y, off, ref = case(pairs, n, v, pairs)
    _, L, _, _, _ = expected((H.double() @ W.double().t()).numpy(), y.numpy(), off.numpy(), ref.double().numpy(), 0.3)
    loss, seq, dH, dW = lce.preference_fwd_bwd(H.cuda(), W.cuda(), y.cuda(), off.cuda(), ref.cuda(), beta=0.3)
    # the head's sums over d may be cut: 2 d 2^-24 of the magnitudes, twice (label and sum)
    mag = float((H.double().abs() @ W.double().abs().t()).max())
    rows = np.diff(off.numpy())
    assert (np.abs(cpu64(seq) - L) <= (rows + 1) * (250 + 4 * d * mag) * 2.0 ** -24 + 2.0 ** -22 * np.abs(L)).all()
    # and what the logits' call, which is checked for itself, gives for these logits (rounded to fp32)
    Z = (H.double() @ W.double().t()).float().cuda()
    l2, _, dZ = lce.preference_logits(Z, y.cuda(), off.cuda(), ref.cuda(), beta=0.3)
    assert abs(loss.item() - l2.item()) <= 1e-4
    want = dZ.double().cpu() @ W.double()
    assert (dH.double().cpu() - want).abs().max() <= 3 * 2.0 ** -8 * want.abs().max()
    assert torch.equal(dW, lce.preference_fwd_bwd(H.cuda(), W.cuda(), y.cuda(), off.cuda(), ref.cuda(), beta=0.3)[3])
