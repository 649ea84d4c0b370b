"""The preference loss over logits and over the head against the fp64 oracle."""
import math

import numpy as np
import pytest
import torch

import linear_cross_entropy_chunked_gb300 as lce
from oracle import answers_oracle as ao
from tests.test_gpu_policy import HALF, TINY, check_gradients, cpu64, logp_bound, rows_like

pytestmark = pytest.mark.gpu


def answers(n, pairs, seed, before=0, behind=0):
    """Offsets of 2 pairs sequences (some empty) in n rows, with rows before and behind them."""
    g = torch.Generator().manual_seed(seed)
    cuts = torch.randint(before, n - behind + 1, (2 * pairs - 1,), generator=g).sort().values
    return torch.cat([torch.tensor([before]), cuts, torch.tensor([n - behind])])


def case(n, v, pairs, seed, ignored=0.3, before=0, behind=0, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(n, v, generator=g) * spread
    y = torch.randint(0, v, (n,), generator=g)
    y[torch.rand(n, generator=g) < ignored] = -100
    return z, y, answers(n, pairs, seed, before, behind)


def reference(z, y, offsets, seed, noise, average=False):
    L = ao.preference(z, y, offsets, average=average)["seq_logprobs"]
    return (torch.from_numpy(L) + noise * torch.randn(len(L), generator=torch.Generator().manual_seed(seed))).float()


def bounds(o, offsets, lb, beta):
    """Bounds of a sequence's log probability, and of a margin's, from that of a row's."""
    rows = np.diff(offsets)
    seq = lb * np.maximum(rows, 1) + 2.0 ** -22 * np.abs(o["seq_logprobs"])
    P = len(rows) // 2
    m = abs(beta) * (seq[:P] + seq[P:]) + 2.0 ** -22 * np.abs(o["margin"])
    return seq, m


def check(loss, seq, o, offsets, lb, beta):
    sb, mb = bounds(o, offsets, lb, beta)
    assert (np.abs(cpu64(seq) - o["seq_logprobs"]) <= sb).all()
    got, want = np.atleast_1d(cpu64(loss)), np.atleast_1d(o["loss"])
    assert (np.abs(got - want) <= mb.max() * (len(mb) if want.size == 1 else 1) + 2.0 ** -21 * (1 + np.abs(want))).all()
    # the slope's sigmoid moves by less than its margin; smoothing leaves the larger part of it
    return mb.max() + 2.0 ** -20


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=str)
@pytest.mark.parametrize("n,v,pairs,layout", [(2, 1, 1, "dense"), (2, 9, 1, "odd"), (40, 33, 3, "padded"), (33, 1000, 16, "dense"),
                                              (25, 4099, 2, "odd"), (9, 50257, 2, "dense"), (5, 128256, 1, "padded"),
                                              (400, 123, 7, "odd")])
def test_logits(n, v, pairs, layout, dtype):
    edge = n // 10
    z, y, off = case(n, v, pairs, n + v, before=edge, behind=edge)
    Z = rows_like(z, layout, dtype)
    for average, e, beta in ((False, 0.0, 0.1), (True, 0.1, 2.0)):
        ref = reference(cpu64(Z), y.numpy(), off.numpy(), n, 0.5 if average else 4.0, average)
        loss, seq, dZ = lce.preference_logits(Z, y.cuda(), off.cuda(), ref.cuda(), beta, e, average)
        o = ao.preference(cpu64(Z), y.numpy(), off.numpy(), ref.numpy(), beta, e, average)
        lb = logp_bound(cpu64(Z), 1.0, v)
        rel = check(loss, seq, o, off.numpy(), lb, beta)
        onehot = np.zeros_like(o["p"])
        onehot[np.flatnonzero(o["ok"]), y.numpy()[o["ok"]]] = 1.0
        scale = np.where(o["ok"] & (o["coef"] != 0), np.abs(o["coef"]) + beta / pairs * rel, 0.0)[:, None]
        bound = ((2 * lb + 2.0 ** -19) * scale + beta / pairs * rel * (scale > 0)) * (o["p"] + onehot)
        bound += HALF[dtype] * (np.abs(o["dZ"]) + bound) + 2 * TINY[dtype] + 1e-37
        assert (np.abs(cpu64(dZ) - o["dZ"]) <= bound).all()
        assert not cpu64(dZ)[o["coef"] == 0].any()
    again = lce.preference_logits(Z, y.cuda(), off.cuda(), ref.cuda(), beta, e, average, inplace=True)
    assert torch.equal(again[0], loss) and torch.equal(again[1], seq) and torch.equal(Z, dZ)


@pytest.mark.parametrize("n,v,ignored", [(5000, 65, 0.5), (2000, 5003, 0.4), (1021, 50257, 0.4)])
def test_many_rows_of_which_some_do_not_count(n, v, ignored):
    g = torch.Generator(device="cuda").manual_seed(n)
    Z = torch.randn(n, v, generator=g, device="cuda").half()
    y = torch.randint(0, v, (n,), generator=g, device="cuda")
    y[torch.rand(n, generator=g, device="cuda") < ignored] = -100
    off = answers(n, 9, n)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    loss, seq, dZ = lce.preference_logits(Z, y, off.cuda(), ws=ws)
    assert lce.read_status(ws) == 0
    lp = torch.log_softmax(Z.double(), 1).gather(1, y.clamp(min=0)[:, None])[:, 0]
    lp = torch.where(y >= 0, lp, 0.0).cpu()
    want = torch.stack([lp[a:b].sum() for a, b in zip(off, off[1:])])
    lb = logp_bound(np.array([[0.0, 14.0]]), 1.0, v)
    assert ((seq.cpu() - want).abs() <= lb * (off[1:] - off[:-1]).clamp(min=1) + 2.0 ** -22 * want.abs()).all()
    assert torch.isfinite(dZ).all() and not dZ[y < 0].any()


@pytest.mark.parametrize("v,dtype", [(600001, torch.float16), (262149, torch.float32)], ids=str)
def test_rows_beyond_the_registers(v, dtype):
    z, y, off = case(4, v, 1, 1, ignored=0.0)
    Z = rows_like(z, "odd", dtype)
    loss, seq, dZ = lce.preference_logits(Z, y.cuda(), off.cuda())
    o = ao.preference(cpu64(Z), y.numpy(), off.numpy())
    lb = logp_bound(cpu64(Z), 1.0, v)
    check(loss, seq, o, off.numpy(), lb, 0.1)
    assert np.abs(cpu64(dZ) - o["dZ"]).max() <= (HALF[dtype] + 8 * lb) * np.abs(o["dZ"]).max() + TINY[dtype]


@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
def test_reductions_and_upstream(reduction):
    z, y, off = case(60, 101, 4, 2)
    Z, P = z.cuda(), 4
    d = torch.randn(P if reduction == "none" else 1, generator=torch.Generator().manual_seed(3))
    loss, seq, dZ = lce.preference_logits(Z, y.cuda(), off.cuda(), reduction=reduction, dloss=d.cuda())
    o = ao.preference(z.numpy(), y.numpy(), off.numpy(), reduction=reduction, dloss=d.numpy())
    assert loss.shape == ((P,) if reduction == "none" else (1,))
    lb = logp_bound(z.double().numpy(), 1.0, 101)
    rel = check(loss, seq, o, off.numpy(), lb, 0.1)
    assert np.abs(cpu64(dZ) - o["dZ"]).max() <= 4 * (rel + lb) * 0.1 * d.abs().max().item()
    l2, s2, none = lce.preference_logits(Z, y.cuda(), off.cuda(), reduction=reduction, grad=False)
    assert none is None and torch.equal(l2, loss) and torch.equal(s2, seq)


def test_extreme_margins():
    z, y, off = case(40, 64, 3, 4, ignored=0.0)
    for shift in (0.0, 1e3, -1e3, 1e30, -1e30):
        ref = torch.full((6,), 0.0)
        ref[:3] = -shift
        loss, _, dZ = lce.preference_logits(z.cuda(), y.cuda(), off.cuda(), ref.cuda(), 0.5)
        o = ao.preference(z.numpy(), y.numpy(), off.numpy(), ref.numpy(), 0.5)
        assert abs(loss.item() - o["loss"]) <= 1e-5 * (1 + abs(o["loss"]))
        assert np.abs(cpu64(dZ) - o["dZ"]).max() <= 1e-5
    z[off[0]] = math.nan   # a NaN in a counting row of the first pair reaches its loss and both gradients
    if off[1] > off[0]:
        loss, seq, dZ = lce.preference_logits(z.cuda(), y.cuda(), off.cuda(), reduction="none")
        assert torch.isnan(loss[0]) and torch.isfinite(loss[1:]).all() and torch.isnan(seq[0])
        assert torch.isnan(dZ[off[0]:off[1]]).all()


def test_offsets_that_do_not_fit_are_flagged():
    z, y, off = case(40, 64, 2, 6, ignored=0.0)
    ws = torch.empty(16384, dtype=torch.uint8, device="cuda")
    for bad in ([0, 30, 20, 35, 40], [0, 10, 20, 30, 41], [-3, 10, 20, 30, 40], [50, 60, 70, 80, 90]):
        _, _, dZ = lce.preference_logits(z.cuda(), y.cuda(), torch.tensor(bad).cuda(), ws=ws)
        assert lce.read_status(ws) == 8 and lce.read_status(ws) == 0
        assert torch.isfinite(dZ).all()
        fixed = np.clip(np.maximum.accumulate(np.clip(bad, 0, 40)), 0, 40)
        o = ao.preference(z.numpy(), y.numpy(), fixed)
        assert np.abs(cpu64(dZ) - o["dZ"]).max() <= 1e-5
    lce.preference_logits(z.cuda(), y.cuda(), off.cuda(), ws=ws)
    assert lce.read_status(ws) == 0


@pytest.mark.parametrize("n,d,v,pairs,chunk", [(2, 8, 3, 1, 1024), (130, 72, 1000, 3, 1024), (300, 264, 1000, 4, 152),
                                               (300, 128, 9001, 5, 128), (500, 64, 700, 2, 64), (64, 512, 300, 8, 7),
                                               (700, 136, 520, 6, 128), (1300, 72, 401, 9, 128), (1100, 64, 300, 4, 1024)])
@pytest.mark.parametrize("mode", ["train", "frozen", "low"])
def test_head(n, d, v, pairs, chunk, mode):
    g = torch.Generator().manual_seed(n)
    H = torch.randn(n, d, generator=g).bfloat16()
    W = (torch.randn(v, d, generator=g) * 2 / math.sqrt(d)).bfloat16()
    edge = n // 12
    _, y, off = case(n, v, pairs, n, before=edge, behind=edge, ignored=0.7 if n > 1000 else 0.3)
    Z = (H.double() @ W.double().t()).numpy()
    if edge:
        H[0] = math.nan   # outside every sequence, with a label that counts
        y[0] = 1
        H[off[1] - 1] = math.nan
        y[off[1] - 1] = -100
    ref = reference(Z, y.numpy(), off.numpy(), 5, 4.0)
    args = [t.cuda() for t in (H, W, y, off, ref)]
    loss, seq, dH, dW = lce.preference_fwd_bwd(*args, beta=0.3, label_smoothing=0.1, chunk=chunk,
                                               compute_dW=mode != "frozen", low_memory=mode == "low")
    o = ao.preference(Z, y.numpy(), off.numpy(), ref.numpy(), 0.3, 0.1)
    Hz = torch.nan_to_num(H.double())
    lb = logp_bound(Z, 1.0, v) + 2 * (2 * d + 8) * 2.0 ** -24 * float((Hz.abs() @ W.double().abs().t()).max())
    rel = check(loss, seq, o, off.numpy(), lb, 0.3)
    check_gradients(dH, dW, Hz, W, o | {"coefs": o["coef"], "y": np.where(o["ok"], y.numpy(), 0),
                                        "coef_err": np.where(o["coef"] != 0, 0.3 / pairs * rel, 0.0)}, lb)
    assert not cpu64(dH)[o["coef"] == 0].any()
    l2, s2, h2, w2 = lce.preference_fwd_bwd(*args, beta=0.3, label_smoothing=0.1, chunk=chunk, gradient=False)
    assert h2 is None and w2 is None and torch.equal(l2, loss) and torch.equal(s2, seq)


@pytest.mark.parametrize("chunk", [1024, 48, 40])
def test_head_accumulates(chunk):
    g = torch.Generator().manual_seed(8)
    H, W = torch.randn(200, 64, generator=g).bfloat16().cuda(), (torch.randn(500, 64, generator=g) * 0.2).bfloat16().cuda()
    _, y, off = case(200, 500, 3, 8)
    y, off = y.cuda(), off.cuda()
    _, _, dH, dW = lce.preference_fwd_bwd(H, W, y, off, chunk=chunk)
    h, w = torch.ones_like(dH), torch.ones_like(dW)
    lce.preference_fwd_bwd(H, W, y, off, chunk=chunk, dH=h, dW=w, accumulate=("dH", "dW"))
    assert (h.float() - 1 - dH.float()).abs().max() <= 2.0 ** -8 * 1.01 + 2.0 ** -8 * dH.float().abs().max()
    assert (w - 1 - dW).abs().max() <= 2.0 ** -21 * (1 + dW.abs().max())


def test_autograd_and_differences():
    g = torch.Generator().manual_seed(11)
    H, W = torch.randn(150, 128, generator=g).bfloat16(), (torch.randn(900, 128, generator=g) * 0.2).bfloat16()
    _, y, off = case(150, 900, 3, 11)
    Z = cpu64(H) @ cpu64(W).T
    ref = reference(Z, y.numpy(), off.numpy(), 1, 3.0)
    h, w = H.cuda().requires_grad_(), W.cuda().requires_grad_()
    loss, seq = lce.linear_preference_loss(h, w, y.cuda(), off.cuda(), ref.cuda(), 0.2, chunk=64)
    assert loss.shape == () and not seq.requires_grad
    gh, gw = torch.autograd.grad(loss * 0.5, (h, w))
    raw = lce.preference_fwd_bwd(H.cuda(), W.cuda(), y.cuda(), off.cuda(), ref.cuda(), 0.2, chunk=64)
    assert torch.equal(gh, (raw[2].float() * 0.5).bfloat16()) and torch.equal(gw, (raw[3] * 0.5).bfloat16())
    o = ao.preference(Z, y.numpy(), off.numpy(), ref.numpy(), 0.2)
    u = np.random.default_rng(0).standard_normal(H.shape)
    step = 1e-5
    up, down = (ao.preference((cpu64(H) + s * u) @ cpu64(W).T, y.numpy(), off.numpy(), ref.numpy(), 0.2)["loss"]
                for s in (step, -step))
    exact = ((o["dZ"] @ cpu64(W)) * u).sum()
    assert abs((up - down) / (2 * step) - exact) <= 1e-6 * max(1.0, abs(exact))
    # without gradients: a reference model's log probabilities, which make the margins zero
    with torch.no_grad():
        _, mine = lce.linear_preference_loss(h, w, y.cuda(), off.cuda())
        l0, _ = lce.linear_preference_loss(h, w, y.cuda(), off.cuda(), mine)
    assert abs(l0.item() - math.log(2)) <= 1e-6


def test_graph_and_stream():
    g = torch.Generator().manual_seed(13)
    H, W = torch.randn(100, 64, generator=g).bfloat16().cuda(), (torch.randn(401, 64, generator=g) * 0.2).bfloat16().cuda()
    _, y, off = case(100, 401, 2, 13)
    y, off = y.cuda(), off.cuda()
    Z = (H @ W.t())[:, :401]

    def step():
        return *lce.preference_fwd_bwd(H, W, y, off, chunk=40), *lce.preference_logits(Z, y, off)
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (14, 15):
        H.copy_(torch.randn(100, 64, generator=g))
        off.copy_(case(100, 401, 2, seed)[2])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, step()))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    side = lce.preference_fwd_bwd(H, W, y, off, chunk=40, stream=s)
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(side, out))
