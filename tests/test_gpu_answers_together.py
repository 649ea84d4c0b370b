"""The losses on answers and the 4-bit layer as they are used together, and the Python calls' refusals of device
tensors that do not fit."""
import math
import threading

import numpy as np
import pytest
import torch

import linear_cross_entropy_chunked_gb300 as lce
from oracle import answers_oracle as ao
from oracle import ops_oracle
from tests.test_gpu_policy import case, check_gradients, cpu64, head, logp_bound, with_coefs
from tests.test_gpu_preference import answers

pytestmark = pytest.mark.gpu


def cut_sums(H, W, temperature=1.0):
    """How far the tensor cores' logits may be off: products of d terms, each step of the sum cut."""
    d = H.shape[1]
    return 2 * (2 * d + 8) * 2.0 ** -24 * float((H.detach().double().abs() @ W.detach().double().abs().t()).max()) / temperature


@pytest.mark.parametrize("n,d,v,group", [(70, 256, 1003, 64), (300, 130, 5003, 32), (9, 512, 777, 128)])
def test_a_policy_step(n, d, v, group):
    # drawn from a head in 4 bits, the loss over the head in 16, the gradients clipped together
    H, W, Z, _, a, _, ref, _ = head(n, d, v, n, ignored=0.0)
    H = (torch.nn.functional.pad(H, (0, -d % 8)) if d % 8 else H).cuda()
    W = (torch.nn.functional.pad(W, (0, -d % 8)) if d % 8 else W).cuda()
    w4 = lce.int4_weight(W, group)
    logits = lce.int4_linear(H, w4)
    want4 = cpu64(H) @ ao.int4_values(w4.q.cpu().numpy(), cpu64(w4.scale), group, H.shape[1]).T
    mass4 = np.abs(cpu64(H)) @ np.abs(ao.int4_values(w4.q.cpu().numpy(), cpu64(w4.scale), group, H.shape[1])).T
    assert (np.abs(cpu64(logits) - want4) <= 2.0 ** -8 * np.abs(want4) + (2 * d + 8) * 2.0 ** -23 * mass4).all()
    u = torch.rand(n, generator=torch.Generator().manual_seed(n)).cuda()
    tokens, old = lce.sample_logits(logits, u, temperature=0.8)
    o4 = ao.log_softmax_of(cpu64(logits), tokens.cpu().numpy(), 0.8)[0]
    assert np.abs(cpu64(old) - o4).max() <= logp_bound(cpu64(logits), 0.8, v) + 2.0 ** -20
    H.requires_grad_()
    W.requires_grad_()
    loss, logprobs = lce.linear_policy_loss(H, W, tokens, a.cuda(), old, old, beta=0.04, temperature=0.8)
    loss.backward()
    Z = cpu64(H) @ cpu64(W).T
    o = ao.policy(Z, tokens.cpu().numpy(), a.numpy(), cpu64(old), cpu64(old), beta=0.04, temperature=0.8)
    lb = logp_bound(Z, 0.8, v) + cut_sums(H, W, 0.8)
    assert np.abs(cpu64(logprobs) - o["logprobs"]).max() <= lb
    assert abs(loss.item() - o["loss"]) <= (2 * lb + 2.0 ** -20) * o["terms"].sum() / n
    check_gradients(H.grad, W.grad, H, W, with_coefs(o, tokens.cpu(), o["mass"]), lb, dw_rounding=2.0 ** -8)
    before = [H.grad.clone(), W.grad.clone()]
    norm = lce.clip_grad_norm([H.grad, W.grad], 0.01)
    want, scaled = ops_oracle.clip([cpu64(b) for b in before], 0.01)
    assert abs(norm.item() - want) <= 19 * 2.0 ** -24 * want
    for got, s in zip((H.grad, W.grad), scaled):
        assert (np.abs(cpu64(got) - s) <= (2.0 ** -8 + 22 * 2.0 ** -24) * np.abs(s) + 1e-40).all()


def test_a_preference_step_against_a_reference_model():
    # the reference's log probabilities from the call without gradients; one head, logits held or not, the same loss
    g = torch.Generator().manual_seed(3)
    H, W = torch.randn(200, 128, generator=g).bfloat16().cuda(), (torch.randn(901, 128, generator=g) * 0.2).bfloat16().cuda()
    _, y, _, _, _, _ = case(200, 901, 3)
    off = answers(200, 5, 3).cuda()
    y = y.cuda()
    older = (W.float() + 0.02 * torch.randn(901, 128, generator=g).cuda()).bfloat16()
    with torch.no_grad():
        _, ref = lce.linear_preference_loss(H, older, y, off)
    h, w = H.clone().requires_grad_(), W.clone().requires_grad_()
    loss, seq = lce.linear_preference_loss(h, w, y, off, ref, 0.2)
    loss.backward()
    o = ao.preference(cpu64(H) @ cpu64(W).T, y.cpu().numpy(), off.cpu().numpy(), cpu64(ref), 0.2)
    lb = (logp_bound(cpu64(H) @ cpu64(W).T, 1.0, 901) + cut_sums(H, W)) * 200
    assert np.abs(cpu64(seq) - o["seq_logprobs"]).max() <= lb + 2.0 ** -22 * np.abs(o["seq_logprobs"]).max()
    assert abs(loss.item() - o["loss"]) <= 0.4 * lb + 1e-6
    Z = (H.float() @ W.float().t()).requires_grad_()
    l2, s2, dZ = lce.preference_logits(Z.detach(), y, off, ref, 0.2)
    assert abs(l2.item() - o["loss"]) <= 0.4 * lb + 1e-6
    dH = dZ.double() @ W.double()
    assert (h.grad.double() - dH).norm() <= 2.0 ** -6 * dH.norm()
    before = w.grad.clone()
    assert lce.clip_grad_norm([h.grad, w.grad], 1e9).item() > 0 and torch.equal(before, w.grad)


def test_margins_of_long_sequences():
    # 64 pairs of two sequences of 256 rows: a row's log probability is off by what the tensor cores cut off the label's
    # logit, up to the mean of it; without that part a margin is less than three quarters as far off
    n, d, v = 64 * 512, 2048, 512
    g = torch.Generator(device="cuda").manual_seed(1)
    H = torch.randn(n, d, generator=g, device="cuda").bfloat16()
    W = (torch.randn(v, d, generator=g, device="cuda") * 3 / math.sqrt(d)).bfloat16()
    Z = H.double() @ W.double().t()
    y = torch.multinomial(torch.softmax(Z, 1).float(), 1, generator=g)[:, 0]
    off = torch.arange(0, n + 1, 256, device="cuda")
    exact = torch.log_softmax(Z, 1).gather(1, y[:, None])[:, 0].view(128, 256).sum(1)
    _, rows = lce.policy_forward(H, W, y, torch.zeros(n, device="cuda"), chunk=8192)
    _, seq, _, _ = lce.preference_fwd_bwd(H, W, y, off, chunk=8192, gradient=False)
    # the margins by their loss (beta = 1, the reference within a few of them), which seq_logprobs' fp32 would round
    ref = exact.float()
    ref[:64] += 0.5
    loss, _, _, _ = lce.preference_fwd_bwd(H, W, y, off, ref, 1.0, chunk=8192, gradient=False, reduction="none")
    with_fix = -torch.log(torch.expm1(loss.double())) - ((exact - ref.double())[:64] - (exact - ref.double())[64:])
    sums = rows.double().view(128, 256).sum(1) - exact
    without = sums[:64] - sums[64:]
    assert (seq.double() - exact).abs().max() <= 256 * 2.0 ** -14
    assert with_fix.pow(2).mean().sqrt() <= 0.75 * without.pow(2).mean().sqrt() + 1e-6


@pytest.mark.parametrize("which", ["policy", "preference"])
def test_the_weight_gradient_in_16_bits(which):
    H, W, _, y, a, old, _, _ = head(700, 136, 901, 4, ignored=0.4)
    dev = [t.cuda() for t in (H, W, y)]
    rest = (a.cuda(), old.cuda()) if which == "policy" else (answers(700, 3, 4).cuda(),)
    call = lce.policy_fwd_bwd if which == "policy" else lce.preference_fwd_bwd
    _, _, dH, dW = call(*dev, *rest)
    _, _, dH16, dW16 = call(*dev, *rest, dW_dtype=torch.bfloat16)
    assert dW16.dtype == torch.bfloat16 and torch.equal(dW16, dW.bfloat16()) and torch.equal(dH16, dH)
    y0 = torch.full_like(dev[2], -100)
    assert not call(dev[0], dev[1], y0, *rest, dW_dtype=torch.bfloat16)[3].any()
    empty = call(dev[0][:0], dev[1], dev[2][:0], *(t[:0] if which == "policy" else torch.zeros_like(t) for t in rest),
                 dW_dtype=torch.bfloat16)
    assert empty[3].dtype == torch.bfloat16 and not empty[3].any()
    for how in (dict(chunk=128), dict(chunk=350, low_memory=True), dict(dW=dW16, accumulate=("dW",)),
                dict(compute_dW=True, dW_dtype=torch.float16)):
        with pytest.raises((RuntimeError, ValueError, TypeError)):
            call(*dev, *rest, **{"dW_dtype": torch.bfloat16, **how})


@pytest.mark.parametrize("chunk", [1024, 64])
def test_backward_twice_and_of_one_input(chunk):
    H, W, _, y, a, old, _, _ = head(300, 64, 501, 6)
    h, w = H.cuda().requires_grad_(), W.cuda().requires_grad_()
    rest = [t.cuda() for t in (y, a, old)]
    loss, _ = lce.linear_policy_loss(h, w, *rest, chunk=chunk)
    first = torch.autograd.grad(loss * 4.0, (h, w), retain_graph=True)
    kept = [t.clone() for t in first]
    (again,) = torch.autograd.grad(loss * 4.0, w, retain_graph=True)
    (gh,) = torch.autograd.grad(loss, h)
    assert all(torch.equal(p, q) for p, q in zip(first, kept))       # what was handed over stays as it was
    # (powers of two: scaled before or after, the same bits)
    assert torch.equal(again, first[1]) and torch.equal(gh * 4.0, first[0])
    loss, _ = lce.linear_policy_loss(h, w, *rest, chunk=chunk)
    gh, gw = torch.autograd.grad(loss, (h, w), create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(gh.float().sum(), h)
    loss, _ = lce.linear_policy_loss(h, w, *rest, chunk=chunk)
    with torch.no_grad():
        w.mul_(1.0)
    with pytest.raises(RuntimeError):   # an input of the saved graph was written to
        loss.backward()


@pytest.mark.parametrize("which", ["policy", "preference"])
def test_captured_steps(which):
    # forward and backward captured together, a backward captured by itself, while an eager graph of other leaves lives
    H, W, _, y, a, old, _, _ = head(300, 64, 501, 8)
    fixed = [t.cuda() for t in (y, a, old)] if which == "policy" else [y.cuda(), answers(300, 3, 8).cuda()]
    call = lce.linear_policy_loss if which == "policy" else lce.linear_preference_loss

    def leaves():
        return H.cuda().requires_grad_(), W.cuda().requires_grad_()
    h0, w0 = leaves()
    eager, _ = call(h0, w0, *fixed)
    want = [t.clone() for t in torch.autograd.grad(eager, (h0, w0), retain_graph=True)]
    side = torch.cuda.Stream()
    h, w = leaves()
    up = torch.tensor(0.5, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(call(h, w, *fixed)[0], (h, w), up)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        loss, _ = call(h, w, *fixed)
        grads = torch.autograd.grad(loss, (h, w), up)
    for factor in (0.5, 2.0, 1.0):
        up.fill_(factor)
        for _ in range(2):
            graph.replay()
        assert all(torch.equal(p, q * factor) for p, q in zip(grads, want))
    h, w = leaves()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        loss, _ = call(h, w, *fixed)
    side.synchronize()
    graph2 = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph2, stream=side):
        grads2 = torch.autograd.grad(loss, (h, w), up)
    for factor in (0.5, 0.5, 2.0):
        up.fill_(factor)
        graph2.replay()
        assert all(torch.equal(p, q * factor) for p, q in zip(grads2, want))
    for p, q in zip(torch.autograd.grad(eager, (h0, w0)), want):
        assert torch.equal(p, q)


@pytest.mark.parametrize("n,v,chunk", [(600, 9, 1024), (600, 9, 128), (90, 3, 64), (300, 40, 128)])
def test_labels_that_many_rows_have(n, v, chunk):
    # lists of more rows than are gone through, rows of weight 0 among them (whose H holds anything where they do not count)
    H, W, Z, y, a, old, _, w = head(n, 72, v, n + v, ignored=0.2)
    w[::3] = 0.0
    H[y < 0] = math.nan
    args = [t.cuda() for t in (H, W, y, a, old)]
    loss, logprobs, dH, dW = lce.policy_fwd_bwd(*args, weights=w.cuda(), chunk=chunk)
    o = ao.policy(np.nan_to_num(Z), y.numpy(), a.numpy(), old.numpy(), weights=w.numpy())
    Hz = torch.nan_to_num(H.double())
    lb = logp_bound(np.nan_to_num(Z), 1.0, v) + cut_sums(Hz, W)
    check_gradients(dH, dW, Hz, W, with_coefs(o, y, o["mass"]), lb)
    assert all(torch.equal(p, q) for p, q in zip(lce.policy_fwd_bwd(*args, weights=w.cuda(), chunk=chunk)[2:], (dH, dW)))


@pytest.mark.parametrize("low_memory", [False, True])
@pytest.mark.parametrize("n,chunk", [(300, 150), (301, 150), (300, 300), (301, 300), (64, 64), (65, 32), (1, 1)])
def test_one_buffer_or_more(n, chunk, low_memory):
    # the largest calls of one contraction, and the smallest of two
    H, W, _, y, a, old, _, _ = head(n, 64, 701, n + chunk)
    h, w = H.cuda().requires_grad_(), W.cuda().requires_grad_()
    rest = [t.cuda() for t in (y, a, old)]
    loss, _ = lce.linear_policy_loss(h, w, *rest, chunk=chunk, low_memory=low_memory)
    loss.backward()
    raw = lce.policy_fwd_bwd(H.cuda(), W.cuda(), *rest, chunk=chunk, low_memory=low_memory)
    assert torch.equal(h.grad, raw[2]) and torch.equal(w.grad, raw[3].bfloat16())
    if n < 2:
        return
    off = answers(n, 1, n).cuda()
    h.grad = w.grad = None
    lce.linear_preference_loss(h, w, rest[0], off, chunk=chunk, low_memory=low_memory)[0].backward()
    raw = lce.preference_fwd_bwd(H.cuda(), W.cuda(), rest[0], off, chunk=chunk, low_memory=low_memory)
    assert torch.equal(h.grad, raw[2]) and torch.equal(w.grad, raw[3].bfloat16())


def test_two_threads_on_two_streams():
    H, W, _, y, a, old, _, _ = head(260, 64, 3001, 12)
    dev = [t.cuda() for t in (H, W, y, a, old)]
    off = answers(260, 3, 1).cuda()
    w4 = lce.int4_weight(dev[1], 32)

    def work():
        Z = lce.int4_linear(dev[0], w4)
        return (*lce.policy_fwd_bwd(*dev), *lce.preference_fwd_bwd(*dev[:3], off), Z, *lce.policy_logits(Z, *dev[2:4]),
                *lce.preference_logits(Z, dev[2], off))
    want = work()
    torch.cuda.synchronize()
    wrong = []

    def run():
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(6):
                got = work()
                torch.cuda.current_stream().synchronize()
                if not all(torch.equal(p, q) for p, q in zip(got, want)):
                    wrong.append(1)
    threads = [threading.Thread(target=run) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_written_tensors_count_as_written():
    H, W, _, y, a, _, _, _ = head(40, 64, 301, 2)
    h, w, y, a = H.cuda(), W.cuda(), y.cuda(), a.cuda()
    off = answers(40, 2, 1).cuda()
    Z = (h @ w.t()).contiguous()
    out = {k: torch.empty(s, device="cuda") for k, s in (("loss", 1), ("logprobs", 40), ("seq_logprobs", 4))}
    dH, dW = torch.empty_like(h), torch.empty(301, 64, device="cuda")
    z4 = torch.empty(40, 304, dtype=torch.bfloat16, device="cuda")[:, :301]
    tensors = [*out.values(), dH, dW, Z, z4]
    before = [t._version for t in tensors]
    lce.policy_fwd_bwd(h, w, y, a, loss=out["loss"], logprobs=out["logprobs"], dH=dH, dW=dW)
    lce.preference_logits(Z, y, off, inplace=True, seq_logprobs=out["seq_logprobs"])
    lce.int4_linear(h, lce.int4_weight(w), out=z4)
    assert all(t._version > b for t, b in zip(tensors, before))


@pytest.mark.parametrize("n", [0, 1, 7, 8, 1000, 4099])
@pytest.mark.parametrize("src", [torch.bfloat16, torch.float16, torch.float32], ids=str)
@pytest.mark.parametrize("dst", [torch.bfloat16, torch.float32], ids=str)
def test_scale(n, src, dst):
    from linear_cross_entropy_chunked_gb300 import _binding as b
    for at in (0, 1):   # rows that start anywhere
        x = torch.randn(n + 8, device="cuda").to(src)
        y = torch.full((n + 8,), math.nan, dtype=dst, device="cuda")
        g = torch.tensor([0.3], device="cuda")
        assert b.lib().lce_scale(x[at:].data_ptr(), b._CE_DTYPES[src], g.data_ptr(), n, y[at:].data_ptr(),
                                 b._CE_DTYPES[dst], torch.cuda.current_stream().cuda_stream) == 0
        assert torch.equal(y[at:at + n], (x[at:at + n].float() * g).to(dst))
        assert torch.isnan(y[:at]).all() and torch.isnan(y[at + n:]).all()


def refuses(call, *args, **how):
    with pytest.raises((ValueError, TypeError)):
        call(*args, **how)


def test_tensors_that_do_not_fit():
    n, d, v = 6, 64, 40
    H, W = torch.randn(n, d, device="cuda").bfloat16(), torch.randn(v, d, device="cuda").bfloat16()
    y, a = torch.zeros(n, dtype=torch.int64, device="cuda"), torch.zeros(n, device="cuda")
    off = torch.tensor([0, 3, 6], device="cuda")
    Z = torch.randn(n, v, device="cuda")
    pol, pre = lce.policy_fwd_bwd, lce.preference_fwd_bwd
    for bad in (a.double(), a[:5], a.cpu(), torch.zeros(2 * n, device="cuda")[::2], a[:, None], None):
        refuses(pol, H, W, y, bad)
        refuses(lce.policy_logits, Z, y, bad)
        if bad is not None:
            for name in ("old_logprobs", "ref_logprobs", "weights"):
                refuses(pol, H, W, y, a, **{name: bad})
    leaf = a.clone().requires_grad_()
    h = H.clone().requires_grad_()
    for name in ("advantages", "old_logprobs", "ref_logprobs", "weights"):
        refuses(lce.linear_policy_loss, h, W, y, **{"advantages": a, name: leaf})
    refuses(lce.linear_preference_loss, h, W, y, off, torch.zeros(2, device="cuda", requires_grad=True))
    refuses(lce.linear_policy_loss, h, W, y, a, reduction="none")
    refuses(pol, H, W, y, a, beta=0.1)
    for bad in (off.int(), off.cpu(), off[:2], off[None], torch.zeros(5, dtype=torch.int64, device="cuda")[:4],
                torch.zeros(6, dtype=torch.int64, device="cuda")[::2]):
        refuses(pre, H, W, y, bad)
        refuses(lce.preference_logits, Z, y, bad)
    refuses(pre, H, W, y, off, torch.zeros(3, device="cuda"))
    for how in (dict(dH=torch.empty(n, d, device="cuda")), dict(dW=torch.empty(v, d, device="cuda").half()),
                dict(loss=torch.empty(2, device="cuda")), dict(ws=torch.empty(16, dtype=torch.uint8, device="cuda")),
                dict(ws=torch.empty(1 << 24, dtype=torch.uint8)), dict(dloss=torch.ones(2, device="cuda")),
                dict(accumulate=("dH",))):
        refuses(pol, H, W, y, a, **how)
        refuses(pre, H, W, y, off, **how)
    refuses(pre, H, W, y, off, gradient=False, dH=torch.empty_like(H))
    for bad in (H.half(), H.float(), H.cpu(), H[:, :63], H[:5]):
        refuses(pol, bad, W, y, a)
        refuses(pre, bad, W, y, off)
    for bad in (Z.double(), Z.cpu(), Z[0], Z.t(), Z.t().contiguous().t()):
        refuses(lce.policy_logits, bad, y, a)
    refuses(lce.policy_logits, Z.clone().requires_grad_(), y, a, inplace=True)
    refuses(lce.policy_logits, Z, y, a, grad=False, inplace=True)
    w4 = lce.int4_weight(W, 32)
    for bad in (H.float(), H.half(), H[0], H.cpu(), H[:, :62], h, H.t()):
        refuses(lce.int4_linear, bad, w4)
    refuses(lce.int4_linear, H, W)
    refuses(lce.int4_linear, H, w4._replace(group=48))
    refuses(lce.int4_linear, H, w4._replace(q=w4.q.contiguous()[:, :31]))
    refuses(lce.int4_linear, H, w4._replace(q=w4.q[1:]))
    refuses(lce.int4_linear, H, w4._replace(scale=w4.scale.half()))
    refuses(lce.int4_linear, H, w4._replace(scale=w4.scale[:, :1]))
    refuses(lce.int4_linear, H, w4, out=torch.empty(n, v, device="cuda"))
    refuses(lce.int4_linear, H, w4, out=torch.empty(n, v + 1, dtype=torch.bfloat16, device="cuda"))
    refuses(lce.int4_weight, W, 48)
    refuses(lce.int4_weight, W, 32, torch.float32)
    refuses(lce.int4_weight, W.double())
