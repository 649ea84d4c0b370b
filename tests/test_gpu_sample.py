"""Token sampling against the fp64 oracle. Tokens are whole numbers and must be equal: the
kernel's cumulative weights are off by about 1e-8 of the row's weight per row of 2^17
tokens in sum, so no border of these few thousand draws is expected to move.

Log-probabilities -x - ls are fp32: x is formed with three roundings (difference, reciprocal,
product), ls by one rounding of its argument and a log of 2 ulp, the sum with one; each at most
2^-24 of its value (a log's ulp 2^-23): together within 2^-22 (x + ls + 1)."""
import numpy as np
import pytest
import torch

import linear_cross_entropy_chunked_gb300 as lce
from oracle import ops_oracle

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
FILTERS = {
    "none": {},
    "temperature": dict(temperature=0.6),
    "hot": dict(temperature=7.5),
    "k1": dict(top_k=1),
    "k": dict(temperature=0.9, top_k=40),
    "p": dict(top_p=0.9),
    "small p": dict(temperature=1.3, top_p=0.05),
    "min": dict(min_p=0.1),
    "k p": dict(temperature=0.8, top_k=300, top_p=0.7),
    "all": dict(temperature=1.1, top_k=50, top_p=0.95, min_p=0.02),
    "greedy": dict(temperature=0.0),
    "p0": dict(top_p=0.0),
    "min1": dict(min_p=1.0),
}


def logits(n, v, seed, dtype, std=2.5):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(n, v, generator=g) * std
    at = torch.randint(0, v, (n, 16), generator=g)
    z.scatter_add_(1, at, 4 + 3 * torch.rand(n, 16, generator=g))
    return z.to(DTYPES[dtype]), torch.rand(n, generator=g)


def check(Z, u, got=None, **settings):
    """Z, u on the host or the device; settings may hold device tensors."""
    if got is None:
        got = lce.sample_logits(Z.cuda(), u.cuda(), **settings)
    tokens, logprobs = (t.cpu().numpy() for t in got)
    host = {k: (s.cpu().double().numpy() if isinstance(s, torch.Tensor) else s) for k, s in settings.items()}
    ref = ops_oracle.sample(Z.double().cpu().numpy(), u.double().cpu().numpy(), **host)
    np.testing.assert_array_equal(tokens, ref["tokens"])
    fin = np.isfinite(ref["logprobs"])
    np.testing.assert_array_equal(logprobs[~fin], ref["logprobs"][~fin].astype(np.float32))
    err = np.abs(logprobs[fin] - ref["logprobs"][fin])
    assert (err <= 2.0 ** -22 * (ref["x"] + ref["ls"] + 1)[fin]).all(), err.max()
    return ref


@pytest.mark.parametrize("name", list(FILTERS))
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("v", [1, 2, 7, 8, 9, 31, 255, 257, 1000, 4097, 32000])
def test_sizes_and_filters(v, dtype, name):
    Z, u = logits(5, v, v * 7 + 1, dtype)
    check(Z, u, **FILTERS[name])


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("name", ["none", "k", "p", "all"])
@pytest.mark.parametrize("v", [50257, 128256, 262144])
def test_large_vocabularies(v, name, dtype):
    Z, u = logits(6, v, v, dtype)
    check(Z, u, **FILTERS[name])


@pytest.mark.parametrize("v,dtype", [(400_003, "fp32"), (1 << 20, "fp32"), (700_001, "bf16"),
                                     (1 << 20, "fp16")])
def test_rows_beyond_shared_memory(v, dtype):
    Z, u = logits(2, v, 3, dtype)
    for name in ("none", "k p", "small p", "greedy"):
        check(Z, u, **FILTERS[name])


@pytest.mark.parametrize("n", [1, 3, 150, 700])
def test_batches(n):
    Z, u = logits(n, 1500, n, "bf16")
    check(Z, u, temperature=0.9, top_p=0.8)


def test_settings_per_row():
    n, v = 96, 3001
    g = torch.Generator().manual_seed(5)
    Z, u = logits(n, v, 17, "bf16")

    def pick(values, dtype):
        return torch.tensor(values, dtype=dtype)[torch.randint(0, len(values), (n,), generator=g)].cuda()
    check(Z, u, temperature=pick([0.0, 0.3, 1.0, 2.0], torch.float32),
          top_k=pick([0, 1, 2, 40, 5000], torch.int32), top_p=pick([1.0, 0.9, 0.3, 0.0], torch.float32),
          min_p=pick([0.0, 0.05, 1.0], torch.float32))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("name", list(FILTERS))
def test_equal_logits(name, dtype):
    # one, two and three distinct values, and both zeros: ties go to the lowest index
    n, v = 4, 5000
    g = torch.Generator().manual_seed(9)
    Z = torch.zeros(n, v)
    Z[1] = torch.randint(0, 2, (v,), generator=g).float()
    Z[2] = torch.randint(0, 3, (v,), generator=g).float() * -0.5
    Z[3] = torch.where(torch.rand(v, generator=g) < 0.5, 0.0, -0.0)
    Z = Z.to(DTYPES[dtype])
    for seed in range(3):
        check(Z, torch.rand(n, generator=g), **FILTERS[name])


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("name", ["none", "k", "p", "all", "greedy"])
def test_masked_logits(name, dtype):
    n, v = 10, 2003
    dt = DTYPES[dtype]
    Z, u = logits(n, v, 23, dtype)
    inf = float("inf")
    Z[0] = -inf                                  # nothing left
    Z[1] = float("nan")
    Z[2] = -inf
    Z[2, v - 1] = -3.0                           # the last token alone
    Z[3, ::2] = -inf
    Z[4, 1::3] = torch.finfo(dt).min
    Z[5] = torch.finfo(dt).min                   # all at the type's lowest value: equal
    Z[6, 5] = inf
    Z[6, 77] = inf                               # share the row
    Z[7, 10:2000] = float("nan")
    Z[8] = torch.finfo(dt).max
    Z[9, :] = -inf
    Z[9, 3] = torch.finfo(dt).min
    check(Z, u, **FILTERS[name])


def test_ends_of_u():
    Z, _ = logits(4, 900, 31, "fp32")
    for f in ({}, dict(top_k=7), dict(top_p=0.5)):
        check(Z, torch.tensor([0.0, 1.0 - 2.0 ** -24, 2.0 ** -149, 0.5]), **f)
        inside = lce.sample_logits(Z.cuda(), torch.tensor([0.0, 1 - 2.0 ** -24] * 2).cuda(), **f)[0]
        outside = lce.sample_logits(Z.cuda(), torch.tensor([-0.5, 1.0, -float("inf"), float("inf")]).cuda(), **f)[0]
        assert torch.equal(inside[[0, 2]], outside[[0, 2]])
        # 1 and beyond: the last kept token
        last = lce.sample_logits(Z.cuda(), torch.full((4,), float("nan")).cuda(), **f)[0]
        assert torch.equal(last[[1, 3]], outside[[1, 3]])


def test_extreme_temperatures():
    Z, u = logits(6, 700, 41, "fp32")
    for t in (1e-6, 1e-3, 50.0, 1e6):
        check(Z, u, temperature=t)
        check(Z, u, temperature=t, top_k=9, top_p=0.9)
    # below the normal numbers: only the largest logit has weight
    tok, lp = lce.sample_logits(Z.cuda(), u.cuda(), temperature=1e-40)
    assert torch.equal(tok.cpu(), Z.argmax(1)) and (lp == 0).all()
    # per row: negative and NaN are greedy
    t = torch.tensor([-1.0, float("nan"), 0.0, -0.0, 1.0, 1.0]).cuda()
    tok = lce.sample_logits(Z.cuda(), u.cuda(), temperature=t)[0]
    assert torch.equal(tok.cpu()[:4], Z.argmax(1)[:4])


def test_strides_and_alignment():
    for dtype in DTYPES:
        base, u = logits(7, 1111, 51, dtype)
        wide = torch.full((7, 1311), float("nan"), dtype=base.dtype, device="cuda")
        for at in (0, 1, 3, 8):
            wide.fill_(float("nan"))
            view = wide[:, at:at + 1111]
            view.copy_(base)
            check(base, u, got=lce.sample_logits(view, u.cuda(), top_p=0.9), top_p=0.9)
        every_other = wide[::2, 2:1113]
        every_other.copy_(base[:4])
        check(base[:4], u[:4], got=lce.sample_logits(every_other, u[:4].cuda()))


def test_draws_follow_the_distribution():
    # 2^16 evenly spread u over one row give each token its share to within 2 draws
    Z, _ = logits(1, 300, 61, "fp32")
    n = 1 << 16
    u = (torch.arange(n) + 0.5) / n
    tok, lp = lce.sample_logits(Z.cuda().expand(n, 300).contiguous(), u.cuda())
    count = torch.bincount(tok.cpu(), minlength=300).double()
    share = torch.softmax(Z[0].double(), 0) * n
    assert (count - share).abs().max() <= 2
    want = torch.log_softmax(Z[0].double(), 0)[tok.cpu()]
    assert (lp.cpu().double() - want).abs().max() < 1e-5


def test_graph_stream_and_repeats():
    Z, u = logits(20, 5003, 71, "bf16")
    Zd, ud = Z.cuda(), u.cuda()
    want = lce.sample_logits(Zd, ud, top_k=30, top_p=0.9)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = lce.sample_logits(Zd, ud, top_k=30, top_p=0.9, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    tok = torch.empty(20, dtype=torch.int64, device="cuda")
    lp = torch.empty(20, device="cuda")
    graphs = []
    for f in (dict(top_k=30, top_p=0.9), dict(temperature=0.0)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            lce.sample_logits(Zd, ud, tokens=tok, logprobs=lp, **f)
        graphs.append((g, f))
    for seed in (72, 73):
        Z2, u2 = logits(20, 5003, seed, "bf16")
        Zd.copy_(Z2)
        ud.copy_(u2)
        for g, f in graphs:
            g.replay()
            check(Z2, u2, got=(tok, lp), **f)


def test_no_rows():
    tok, lp = lce.sample_logits(torch.empty(0, 100, device="cuda"), torch.empty(0, device="cuda"))
    assert tok.shape == (0,) and lp.shape == (0,)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("std", [0.01, 0.3, 1.0, 6.0, 40.0])
def test_flat_and_peaked_rows(std, dtype):
    # cuts among few and among tens of thousands of tokens, near the largest logit and far from it
    for v in (3000, 60000):
        Z, u = logits(3, v, int(std * 100) + v, dtype, std=std)
        Z[0] = (torch.randn(v, generator=torch.Generator().manual_seed(v)) * std).to(Z.dtype)
        for f in (dict(top_p=0.999), dict(top_p=0.5), dict(top_k=128), dict(top_k=129), dict(top_k=2000, top_p=0.97),
                  dict(top_k=v - 1), dict(top_k=60, top_p=0.9, min_p=0.3)):
            check(Z, u, **f)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_ties_around_the_cut(dtype):
    # more equal logits than the cut leaves room for, few and many
    for v, n_top, n_tie in ((2000, 3, 40), (70000, 5, 100), (70000, 30, 5000), (70000, 0, 70000)):
        Z = torch.full((3, v), -4.0)
        Z[1] = torch.randn(v, generator=torch.Generator().manual_seed(1)) - 4
        at = torch.randperm(v, generator=torch.Generator().manual_seed(2))
        Z[:, at[:n_tie]] = 1.5
        Z[:, at[:n_top]] = 3.0
        Z = Z.to(DTYPES[dtype])
        u = torch.tensor([0.999, 0.3, 0.7])
        for f in (dict(top_k=n_top + 1), dict(top_k=n_top + n_tie // 2 + 1), dict(top_p=0.5), dict(top_p=0.9),
                  dict(top_k=max(1, n_top), min_p=0.5)):
            check(Z, u, **f)


@pytest.mark.parametrize("kw", [{}, {"top_k": 50}, {"top_k": 5000}, {"top_p": 0.9}, {"top_k": 3000, "top_p": 0.8},
                                {"min_p": 0.01}, {"temperature": 0.0}])
@pytest.mark.parametrize("n,v,dtype", [(400, 50257, torch.float32), (330, 100003, torch.bfloat16),
                                       (170, 60000, torch.float16)])
def test_a_row_is_drawn_the_same_in_any_batch(n, v, dtype, kw):
    # few rows are split over many CTAs and stay in shared memory, many are read again
    g = torch.Generator(device="cuda").manual_seed(n)
    Z = (torch.randn(n, v, device="cuda", generator=g) * 2).to(dtype)
    Z[1, 7] = float("nan")
    Z[2, ::2] = -float("inf")
    Z[3, ::3] = -0.0
    u = torch.rand(n, device="cuda", generator=g)
    tokens, logprobs = lce.sample_logits(Z, u, **kw)
    for a in (0, n // 2, n - 5):
        t, lp = lce.sample_logits(Z[a:a + 5], u[a:a + 5], **kw)
        assert torch.equal(t, tokens[a:a + 5]) and torch.equal(lp, logprobs[a:a + 5])
