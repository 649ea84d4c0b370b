"""The policy loss over logits and over the head against the fp64 oracle."""
import math

import numpy as np
import pytest
import torch

import linear_cross_entropy_chunked_gb300 as lce
from oracle import answers_oracle as ao

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -149}


def cpu64(t):
    return t.detach().double().cpu().numpy()


def rows_like(z, layout, dtype):
    """z [N, V] as a device tensor: dense rows, padded rows with NaN behind them, or dense from an odd element on."""
    n, v = z.shape
    if layout == "dense":
        return z.to(dtype).cuda()
    if layout == "padded":
        buf = torch.full((n, (v + 23) // 8 * 8), math.nan, dtype=dtype)
        buf[:, :v] = z.to(dtype)
        return buf.cuda()[:, :v]
    buf = torch.full((n * v + 9,), math.nan, dtype=dtype, device="cuda")
    out = buf[3:3 + n * v].view(n, v)
    out.copy_(z.to(dtype))
    return out


def case(n, v, seed, spread=3.0, ignored=0.3):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(n, v, generator=g) * spread
    y = torch.randint(0, v, (n,), generator=g)
    y[torch.rand(n, generator=g) < ignored] = -100
    logp = ao.log_softmax_of(z.double().numpy(), y.numpy())[0]
    old = torch.from_numpy(logp).float() + 0.25 * torch.randn(n, generator=g)
    ref = torch.from_numpy(logp).float() + 0.4 * torch.randn(n, generator=g)
    return z, y, torch.randn(n, generator=g), old, ref, torch.rand(n, generator=g) + 0.1


def logp_bound(z, temperature, v):
    """How far fp32 log probabilities may be off: the distances from the largest logit (up to `far`)
    are rounded three times, a sum of v positive terms goes through at most 32 + log2 v
    additions per term, ex2 is off by 2^-22."""
    far = float(np.ptp(np.where(np.isfinite(z), z, 0.0), axis=1).max()) / temperature
    return (3 * far * 1.4427 + 2 * (2 + 40 + math.log2(v + 1)) + 8 + math.log(v + 1)) * 2.0 ** -24


def check(Z, y, loss, logprobs, dZ, o, temperature, dtype):
    lb = logp_bound(cpu64(Z), temperature, Z.shape[1])
    assert np.abs(cpu64(logprobs) - o["logprobs"]).max(initial=0.0) <= lb
    # a row's loss and coefficient: terms that move by lb relative (their exponent does), and a dozen roundings
    rel = 2 * lb + 12 * 2.0 ** -24
    n = max(1, o["ok"].sum())
    got, want = np.atleast_1d(cpu64(loss)), np.atleast_1d(o["loss"])
    terms = o["terms"] if want.size == Z.shape[0] and want.size > 1 else np.atleast_1d(o["terms"].sum())
    if terms.size == 1 and o.get("reduction") == "mean":
        terms = terms / n
    assert (np.abs(got - want) <= rel * terms + 2.0 ** -23 * np.abs(want) + 1e-30).all(), (got, want)
    if dZ is None:
        return
    assert dZ.dtype == dtype and dZ.shape == Z.shape
    onehot = np.zeros_like(o["p"])
    onehot[np.flatnonzero(o["ok"]), y.cpu().numpy()[o["ok"]]] = 1.0
    bound = 2 * rel * o["mass"][:, None] * (o["p"] + onehot) + HALF[dtype] * np.abs(o["dZ"]) + 2 * TINY[dtype] + 1e-37
    err = np.abs(cpu64(dZ) - o["dZ"])
    assert (err <= bound).all(), float((err / bound).max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=str)
@pytest.mark.parametrize("n,v,layout", [(1, 1, "dense"), (3, 7, "dense"), (5, 8, "odd"), (7, 33, "padded"), (17, 1000, "dense"),
                                        (6, 4099, "odd"), (33, 4099, "dense"), (9, 50257, "dense"), (4, 50257, "odd"),
                                        (3, 128256, "padded"), (200, 777, "odd")])
def test_logits(n, v, layout, dtype):
    z, y, a, old, ref, w = case(n, v, 7 * n + v)
    Z = rows_like(z, layout, dtype)
    how = dict(clip_low=0.2, clip_high=0.3, beta=0.1, temperature=0.8)
    loss, logprobs, dZ = lce.policy_logits(Z, y.cuda(), a.cuda(), old.cuda(), ref.cuda(), w.cuda(), **how)
    o = ao.policy(cpu64(Z), y.numpy(), a.numpy(), old.numpy(), ref.numpy(), w.numpy(), **how) | {"reduction": "mean"}
    assert dZ.stride(0) == Z.stride(0) or n == 1
    check(Z, y, loss, logprobs, dZ, o, 0.8, dtype)
    # the same bits again, in place, and nothing beside the rows touched
    again = lce.policy_logits(Z, y.cuda(), a.cuda(), old.cuda(), ref.cuda(), w.cuda(), inplace=True, **how)
    assert torch.equal(again[0], loss) and torch.equal(again[1], logprobs) and torch.equal(Z, dZ)
    if layout != "dense":
        whole = torch.as_strided(Z, (Z.untyped_storage().nbytes() // Z.element_size(),), (1,), 0)
        inside = torch.zeros_like(whole, dtype=torch.bool)
        torch.as_strided(inside, Z.shape, Z.stride(), Z.storage_offset()).fill_(True)
        assert torch.isnan(whole[~inside]).all()


@pytest.mark.parametrize("v,dtype", [(524295, torch.bfloat16), (600001, torch.float16), (262149, torch.float32)], ids=str)
@pytest.mark.parametrize("layout", ["dense", "odd"])
def test_rows_beyond_the_registers(v, dtype, layout):
    z, y, a, old, _, _ = case(3, v, v, ignored=0.2)
    y[0], y[2] = v - 1, -100
    Z = rows_like(z, layout, dtype)
    loss, logprobs, dZ = lce.policy_logits(Z, y.cuda(), a.cuda(), old.cuda(), reduction="sum")
    o = ao.policy(cpu64(Z), y.numpy(), a.numpy(), old.numpy(), reduction="sum")
    check(Z, y, loss, logprobs, dZ, o, 1.0, dtype)


@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
@pytest.mark.parametrize("n", [1, 5, 300])
def test_reductions_and_upstream(n, reduction):
    z, y, a, old, ref, w = case(n, 501, n)
    Z = rows_like(z, "dense", torch.float32)
    g = torch.Generator().manual_seed(1)
    d = torch.randn(n if reduction == "none" else 1, generator=g)
    for o_, w_ in ((old, None), (None, w), (old, w)):
        kw = dict(old_logprobs=None if o_ is None else o_.cuda(), weights=None if w_ is None else w_.cuda())
        loss, logprobs, dZ = lce.policy_logits(Z, y.cuda(), a.cuda(), dloss=d.cuda(), reduction=reduction, **kw)
        o = ao.policy(cpu64(Z), y.numpy(), a.numpy(), None if o_ is None else o_.numpy(), None,
                      None if w_ is None else w_.numpy(), reduction=reduction, dloss=d.numpy()) | {"reduction": reduction}
        check(Z, y, loss, logprobs, dZ, o, 1.0, torch.float32)
        l2, lp2, none = lce.policy_logits(Z, y.cuda(), a.cuda(), reduction=reduction, grad=False, **kw)
        assert none is None and torch.equal(l2, loss) and torch.equal(lp2, logprobs)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
def test_masked_logits_and_rows_that_do_not_count(dtype):
    v = 40003
    z, y, a, old, ref, w = case(12, v, 3, ignored=0.0)
    z[0, 1:] = -math.inf               # one token left
    y[0] = 0
    z[1, 20000:] = -math.inf           # whole CTAs of nothing
    y[1] = 5
    z[2] = torch.finfo(dtype).min      # every token alike
    z[3, :] = math.nan                 # rows that do not count hold anything
    y[3] = -100
    z[4, 3] = math.inf
    y[4] = -100
    y[5] = v                           # outside: does not count, and is flagged
    a[6] = 0.0
    old[6] = -1e4                      # the ratio overflows
    z[7, 100:] = -math.inf
    y[7] = 30000                       # the label itself is masked
    Z = rows_like(z, "dense", dtype)
    ws = torch.empty(4096, dtype=torch.uint8, device="cuda")
    loss, logprobs, dZ = lce.policy_logits(Z, y.cuda(), a.cuda(), old.cuda(), ws=ws, reduction="none")
    assert lce.read_status(ws) == 4 and lce.read_status(ws) == 0
    with np.errstate(all="ignore"):
        o = ao.policy(cpu64(Z), y.numpy(), a.numpy(), old.numpy(), reduction="none")
    lp, l, d = cpu64(logprobs), cpu64(loss), cpu64(dZ)
    assert lp[0] == 0 and abs(lp[2] + math.log(v)) <= 1e-5
    assert (lp[[3, 4, 5]] == 0).all() and (l[[3, 4, 5]] == 0).all() and (d[[3, 4, 5]] == 0).all()
    assert l[6] == 0 and (d[6] == 0).all()
    assert lp[7] == -math.inf and np.isfinite(d[7]).all()
    keep = [0, 1, 2, 8, 9, 10, 11]
    sub = {k: v_[keep] for k, v_ in o.items()}
    check(Z[keep], y[keep], loss[keep], logprobs[keep], dZ[keep], sub, 1.0, dtype)
    # a counting row without any token, or with a NaN, says so
    z[8] = -math.inf
    z[9, 7] = math.nan
    loss, logprobs, dZ = lce.policy_logits(rows_like(z, "dense", dtype), y.cuda(), a.cuda(), old.cuda())
    assert torch.isnan(logprobs[[8, 9]]).all() and torch.isnan(dZ[[8, 9]]).all() and torch.isnan(loss).all()
    assert np.array_equal(cpu64(dZ[10:]) * 9, cpu64(dZ[10:]) * 9)


@pytest.mark.parametrize("n,v,ignored", [(5000, 65, 0.5), (3001, 33, 0.95), (2000, 5003, 0.4), (1021, 50257, 0.4)])
def test_many_rows_of_which_some_do_not_count(n, v, ignored):
    # (several rows per CTA, in every order of counting ones and others: no wait runs out)
    g = torch.Generator(device="cuda").manual_seed(n)
    Z = torch.randn(n, v, generator=g, device="cuda").half()
    y = torch.randint(0, v, (n,), generator=g, device="cuda")
    y[torch.rand(n, generator=g, device="cuda") < ignored] = -100
    a = torch.randn(n, generator=g, device="cuda")
    ws = torch.empty(65536, dtype=torch.uint8, device="cuda")
    loss, logprobs, dZ = lce.policy_logits(Z, y, a, ws=ws)
    assert lce.read_status(ws) == 0
    z, ok = Z.double(), y >= 0
    lp = torch.log_softmax(z, 1)
    want = torch.where(ok, lp.gather(1, y.clamp(min=0)[:, None])[:, 0], 0.0)
    lb = logp_bound(np.array([[0.0, 14.0]]), 1.0, v)
    assert (logprobs - want).abs().max() <= lb
    p = lp.exp_()
    p[ok, y[ok]] -= 1.0
    p *= torch.where(ok, a.double() / ok.sum(), 0.0)[:, None]
    bound = 2.0 ** -11 * p.abs() + 2 * TINY[torch.float16] + 4 * lb * (a.double().abs() / ok.sum())[:, None] * p.abs().clamp(min=1e-9)
    assert ((dZ.double() - p).abs() <= bound + 4 * lb * a.abs().max() / ok.sum()).all()
    assert not dZ[~ok].any()


def test_no_rows_and_no_counting_rows():
    f = torch.empty(0, device="cuda")
    loss, logprobs, dZ = lce.policy_logits(torch.empty(0, 50, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda"), f)
    assert loss.item() == 0 and logprobs.shape == (0,) and dZ.shape == (0, 50)
    z, y, a, old, _, _ = case(70, 301, 5, ignored=2.0)
    loss, logprobs, dZ = lce.policy_logits(z.cuda() * math.nan, y.cuda(), a.cuda(), old.cuda())
    assert loss.item() == 0 and not logprobs.any() and not dZ.any()
    H = torch.full((70, 64), math.nan, dtype=torch.bfloat16, device="cuda")
    W = torch.randn(301, 64, device="cuda").bfloat16()
    loss, logprobs, dH, dW = lce.policy_fwd_bwd(H, W, y.cuda(), a.cuda(), old.cuda(), chunk=32)
    assert loss.item() == 0 and not logprobs.any() and not dH.any() and not dW.any()


def head(n, d, v, seed, ignored=0.3):
    g = torch.Generator().manual_seed(seed)
    H = torch.randn(n, d, generator=g).bfloat16()
    W = (torch.randn(v, d, generator=g) * 2 / math.sqrt(d)).bfloat16()
    Z = H.double() @ W.double().t()
    _, y, a, _, _, w = case(n, v, seed, ignored=ignored)
    logp = ao.log_softmax_of(Z.numpy(), y.numpy())[0]
    old = (torch.from_numpy(logp) + 0.25 * torch.randn(n, generator=g)).float()
    ref = (torch.from_numpy(logp) + 0.4 * torch.randn(n, generator=g)).float()
    return H, W, Z.numpy(), y, a, old, ref, w


def check_gradients(dH, dW, H, W, o, lb, out_rounding=2.0 ** -8, dw_rounding=0.0):
    """G is rounded twice to bf16 (as exp(z - slab maximum), then scaled), but for the onehot's part, whose second
    rounding is made up for (in dW for labels that 8 rows or fewer have); sums in fp32 of up to 2^17 terms, of
    which fewer than 2^8 follow one another; dH is rounded once more, dW is fp32. coef_err: how far the coefficients
    themselves may be off."""
    step, rel = 2.0 ** -8, 4 * lb + 2.0 ** -14
    mass = np.abs(o["coefs"])[:, None] * o["p"]
    onehot = np.zeros_like(mass)
    onehot[np.arange(len(o["y"])), o["y"]] = np.abs(o["coefs"]) * o["ok"]
    ones = (onehot != 0) * o.get("coef_err", np.zeros(len(mass)))[:, None]
    off = rel * (mass + onehot) + ones + (ones.sum(1, keepdims=True) * o["p"])
    h, w = cpu64(H), cpu64(W)
    want = o["dZ"] @ w
    bound = (2 * step * mass + off) @ np.abs(w)
    assert (np.abs(cpu64(dH) - want) <= bound + out_rounding * (np.abs(want) + bound) + 1e-30).all()
    if dW is not None:
        want = o["dZ"].T @ h
        many = np.bincount(o["y"][o["ok"]], minlength=mass.shape[1])[:, None] > 8
        bound = (2 * step * mass + off).T @ np.abs(h) + step * many * (onehot.T @ np.abs(h))
        assert (np.abs(cpu64(dW) - want) <= bound + dw_rounding * (np.abs(want) + bound) + 1e-30).all()


def with_coefs(o, y, scale):
    return o | {"coefs": scale, "y": np.where(o["ok"], y.numpy(), 0)}


@pytest.mark.parametrize("n,d,v,chunk", [(1, 8, 3, 1024), (5, 64, 129, 1024), (130, 72, 1000, 64), (300, 264, 1000, 128),
                                         (257, 128, 9001, 104), (64, 512, 300, 7), (700, 136, 520, 128)])
@pytest.mark.parametrize("mode", ["train", "frozen", "low"])
def test_head(n, d, v, chunk, mode):
    H, W, Z, y, a, old, ref, w = head(n, d, v, n + d)
    if n > 4:
        y[2] = -100
        H[2] = math.nan   # a row that does not count holds anything
        Z[2] = 0
    how = dict(clip_low=0.1, clip_high=0.3, beta=0.05, temperature=0.7)
    loss, logprobs, dH, dW = lce.policy_fwd_bwd(
        H.cuda(), W.cuda(), y.cuda(), a.cuda(), old.cuda(), ref.cuda(), w.cuda(), chunk=chunk,
        compute_dW=mode != "frozen", low_memory=mode == "low", **how)
    o = ao.policy(Z, y.numpy(), a.numpy(), old.numpy(), ref.numpy(), w.numpy(), **how)
    # products of d terms in fp32, some of which may be cut, not rounded, on the way: 2 d 2^-24 of the sum of magnitudes
    Hz = torch.nan_to_num(H.double())
    lb = logp_bound(Z, 0.7, v) + 2 * (2 * d + 8) * 2.0 ** -24 * float((Hz.abs() @ W.double().abs().t()).max()) / 0.7
    assert np.abs(cpu64(logprobs) - o["logprobs"]).max() <= lb
    assert abs(loss.item() - o["loss"]) <= (2 * lb + 2.0 ** -20) * o["terms"].sum() / max(1, o["ok"].sum())
    check_gradients(dH, dW, torch.nan_to_num(H), W, with_coefs(o, y, o["mass"]), lb)
    assert dW is not None or mode == "frozen"
    l2, lp2 = lce.policy_forward(H.cuda(), W.cuda(), y.cuda(), a.cuda(), old.cuda(), ref.cuda(), w.cuda(), chunk=chunk, **how)
    assert torch.equal(lp2, logprobs) and torch.equal(l2, loss)


@pytest.mark.parametrize("ignored", [0.0, 0.5, 0.97, 2.0])
@pytest.mark.parametrize("n,chunk", [(300, 1024), (700, 128), (1000, 64), (1000, 192), (513, 512), (257, 64)])
@pytest.mark.parametrize("mode", ["train", "frozen", "low"])
def test_rows_brought_together(n, chunk, mode, ignored):
    # more rows than a tile has: those that count come first, whole chunks may be empty, the last k block of the
    # weight's contraction is part rows and part nothing; what rows that do not count hold stays there
    d, v = 72, 333
    H, W, Z, y, a, old, ref, w = head(n, d, v, n + chunk, ignored=ignored)
    H[y < 0] = math.nan
    if ignored == 0.97:
        y[: n // 2] = -100
    how = dict(beta=0.05, temperature=0.9)
    args = [t.cuda() for t in (H, W, y, a, old, ref, w)]
    kw = dict(chunk=chunk, compute_dW=mode != "frozen", low_memory=mode == "low")
    loss, logprobs, dH, dW = lce.policy_fwd_bwd(*args, **how, **kw)
    Z = np.nan_to_num(Z)
    o = ao.policy(Z, y.numpy(), a.numpy(), old.numpy(), ref.numpy(), w.numpy(), **how)
    Hz = torch.nan_to_num(H.double())
    lb = logp_bound(Z, 0.9, v) + 2 * (2 * d + 8) * 2.0 ** -24 * float((Hz.abs() @ W.double().abs().t()).max()) / 0.9
    assert np.abs(cpu64(logprobs) - o["logprobs"]).max() <= lb
    assert abs(loss.item() - o["loss"]) <= (2 * lb + 2.0 ** -20) * o["terms"].sum() / max(1, o["ok"].sum())
    check_gradients(dH, dW, Hz, W, with_coefs(o, y, o["mass"]), lb)
    assert not dH[y < 0].any()
    again = lce.policy_fwd_bwd(*args, **how, **kw)
    assert all(p is q or torch.equal(p, q) for p, q in zip(again, (loss, logprobs, dH, dW)))
    rows, lp, _, _ = lce.policy_fwd_bwd(*args, **how, **kw, reduction="none")
    assert torch.equal(lp, logprobs) and not rows[y < 0].any()
    assert abs(rows.double().sum().item() / max(1, o["ok"].sum()) - o["loss"]) <= 1e-5 * (1 + o["terms"].sum())
    assert torch.equal(lce.policy_forward(*args, **how, chunk=chunk)[1], logprobs)
    if mode == "train":
        more = [torch.ones(n, d, dtype=torch.bfloat16, device="cuda"), torch.ones_like(dW)]
        lce.policy_fwd_bwd(*args, **how, chunk=chunk, dH=more[0], dW=more[1], accumulate=("dH", "dW"))
        # every contraction (of a chunk or two) adds to values near 1, each time within 2^-24 of them, here and
        # once more in this comparison
        adds = -(-n // chunk) + 2
        assert (more[1] - 1 - dW).abs().max() <= adds * 2.0 ** -24 * (1 + 2 * dW.abs().max())
        assert (more[0].float() - 1 - dH.float()).abs().max() <= 2.0 ** -8 * (1.01 + dH.float().abs().max())
        assert (more[0][y < 0] == 1).all()


@pytest.mark.parametrize("n,chunk", [(90, 1024), (300, 64)])
def test_head_accumulates_and_reduces(n, chunk):
    H, W, Z, y, a, old, ref, w = head(n, 64, 700, n)
    dev = [t.cuda() for t in (H, W, y, a, old)]
    _, _, dH, dW = lce.policy_fwd_bwd(*dev, chunk=chunk)
    more = [torch.ones_like(dH), torch.ones_like(dW)]
    lce.policy_fwd_bwd(*dev, chunk=chunk, dH=more[0], dW=more[1], accumulate=("dH", "dW"))
    assert (more[0].float() - 1 - dH.float()).abs().max() <= 2.0 ** -8 * 1.01 + 2.0 ** -8 * dH.float().abs().max()
    assert (more[1] - 1 - dW).abs().max() <= 2.0 ** -22 * (1 + dW.abs().max())
    d = torch.rand(n, generator=torch.Generator().manual_seed(2)) - 0.5
    loss, logprobs, dH, dW = lce.policy_fwd_bwd(*dev, chunk=chunk, reduction="none", dloss=d.cuda())
    o = ao.policy(Z, y.numpy(), a.numpy(), old.numpy(), reduction="none", dloss=d.numpy())
    assert np.abs(cpu64(loss) - o["loss"]).max() <= 1e-4 * o["terms"].max()
    check_gradients(dH, dW, H, W, with_coefs(o, y, o["mass"]), 1e-4)


def test_autograd_and_differences():
    H, W, Z, y, a, old, ref, w = head(150, 128, 900, 9, ignored=0.2)
    dev = [t.cuda() for t in (y, a, old, ref)]
    kw = dict(old_logprobs=dev[2], ref_logprobs=dev[3], beta=0.1, chunk=64)
    h, wt = H.cuda().requires_grad_(), W.cuda().requires_grad_()
    loss, logprobs = lce.linear_policy_loss(h, wt, dev[0], dev[1], **kw)
    assert loss.shape == () and not logprobs.requires_grad
    gh, gw = torch.autograd.grad(3.0 * loss, (h, wt))
    raw = lce.policy_fwd_bwd(H.cuda(), W.cuda(), dev[0], dev[1], **kw)
    assert torch.equal(gh, (raw[2].float() * 3).bfloat16()) and torch.equal(gw, (raw[3] * 3).bfloat16())
    # along a direction of the weight: the difference of the oracle's losses
    o = ao.policy(Z, y.numpy(), a.numpy(), old.numpy(), ref.numpy(), beta=0.1)
    g = np.random.default_rng(0).standard_normal(W.shape)
    step = 1e-5
    up, down = (ao.policy(cpu64(H) @ (cpu64(W) + s * g).T, y.numpy(), a.numpy(), old.numpy(), ref.numpy(), beta=0.1)["loss"]
                for s in (step, -step))
    along = (up - down) / (2 * step)
    exact = ((o["dZ"].T @ cpu64(H)) * g).sum()
    assert abs(along - exact) <= 1e-5 * np.abs(o["dZ"].T @ cpu64(H)).max() * math.sqrt(g.size)
    got = (cpu64(raw[3]) * g).sum()
    assert abs(got - exact) <= 2.0 ** -7 * np.linalg.norm(o["dZ"].T @ cpu64(H)) * 4
    # a frozen head, a frozen body, and no gradient at all
    loss2, _ = lce.linear_policy_loss(h, W.cuda(), dev[0], dev[1], **kw)
    (g2,) = torch.autograd.grad(loss2, h)
    assert torch.equal(loss2, loss) and (g2.float() - raw[2].float()).abs().max() <= 2.0 ** -7 * raw[2].float().abs().max()
    (g3,) = torch.autograd.grad(lce.linear_policy_loss(H.cuda(), wt, dev[0], dev[1], **kw)[0], wt)
    assert torch.equal(g3, raw[3].bfloat16())
    with torch.no_grad():
        assert torch.equal(lce.linear_policy_loss(h, wt, dev[0], dev[1], **kw)[0], loss)


def test_graph_stream_and_reference_policy():
    # captured once, replayed on new inputs; and on a stream of its own
    H, W, _, y, a, old, _, _ = head(96, 64, 1001, 21)
    buf = [t.cuda() for t in (H, W, y, a, old)]

    def step():
        loss, logprobs, dH, dW = lce.policy_fwd_bwd(*buf, chunk=40)
        return loss, logprobs, dH, dW, *lce.policy_logits(dH, buf[2] % 64, buf[3])
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (22, 23):
        new = head(96, 64, 1001, seed)
        for b, t in zip(buf, (new[0], new[1], new[3], new[4], new[5])):
            b.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, step()))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    side = lce.policy_fwd_bwd(*buf, chunk=40, stream=s)
    side_z = lce.policy_logits(buf[0], buf[2] % 64, buf[3], stream=s)
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(side, out)) and torch.isfinite(side_z[2].float()).all()
