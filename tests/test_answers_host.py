"""Host-side tests of the losses on answers and the 4-bit linear layer (no GPU): argument errors of the C ABI,
refusals of the Python calls, and the fp64 oracle against independent definitions. Pointer arguments are
fake addresses that the library must reject before it touches the device."""
import ctypes
import math

import numpy as np
import pytest
import torch

import linear_cross_entropy_chunked_gb300 as lce
from oracle import answers_oracle as ao

OK, INVALID, ALIGN, WORKSPACE, UNSUPPORTED = 0, 1, 2, 3, 7
FAKE = 0x10000000
FAR = FAKE + (1 << 30)


@pytest.fixture(scope="module")
def L():
    try:
        lce.build()
    except RuntimeError as e:  # no nvcc here
        pytest.skip(str(e))
    return lce.lib()


POLICY = dict(adv=FAKE, old=None, ref=None, w=None, lo=0.2, hi=0.2, beta=0.0, t=1.0)


def policy_logits(L, Z=FAKE, dtype=0, ld=1000, y=FAKE, N=4, V=1000, red=0, dloss=None, loss=FAKE, lp=FAKE, dZ=FAR, ws=FAKE,
                  nbytes=2048, **how):
    h = POLICY | how
    return L.lce_policy_logits(Z, dtype, ld, y, h["adv"], h["old"], h["ref"], h["w"], h["lo"], h["hi"], h["beta"],
                               h["t"], dloss, N, V, -100, red, loss, lp, dZ, ws, nbytes, None)


BAD_POLICY = [(dict(adv=None), INVALID), (dict(lo=-0.1), INVALID), (dict(lo=1.5), INVALID), (dict(lo=math.nan), INVALID),
              (dict(hi=-0.1), INVALID), (dict(hi=math.inf), INVALID), (dict(beta=-1.0), INVALID), (dict(beta=math.nan), INVALID),
              (dict(beta=0.1), INVALID), (dict(t=0.0), INVALID), (dict(t=-1.0), INVALID), (dict(t=math.inf), INVALID),
              (dict(t=1e-45), INVALID), (dict(t=5e-20), INVALID), (dict(adv=FAKE + 2), ALIGN), (dict(old=FAKE + 1), ALIGN), (dict(ref=FAKE + 2), ALIGN),
              (dict(w=FAKE + 3), ALIGN), (dict(lp=None), INVALID), (dict(lp=FAKE + 2), ALIGN)]


@pytest.mark.parametrize("how,want", BAD_POLICY, ids=str)
def test_policy_arguments(L, how, want):
    assert policy_logits(L, **how) == want
    h = POLICY | {"lp": FAKE} | how
    pol = (h["adv"], h["old"], h["ref"], h["w"], h["lo"], h["hi"], h["beta"], h["t"])
    assert L.lce_policy_fwd_bwd(FAKE, FAKE, FAKE, *pol, None, 4, 64, 100, -100, 4, 0, 0, FAKE, h["lp"], FAKE, FAKE, FAKE,
                                1 << 30, None) == want
    assert L.lce_policy_forward(FAKE, FAKE, FAKE, *pol, 4, 64, 100, -100, 4, 0, FAKE, h["lp"], FAKE, 1 << 30, None) == want


def test_16_bit_weight_gradients(L):
    # one contraction of a trained weight that is not added to (refused before the device is asked)
    pol = tuple(POLICY.values())

    def policy(N=4, chunk=4, flags=32):
        return L.lce_policy_fwd_bwd(FAKE, FAKE, FAKE, *pol, None, N, 64, 100, -100, chunk, 0, flags, FAKE, FAKE, FAKE, FAKE, FAKE,
                                    1 << 40, None)

    def preference(N=4, chunk=4, flags=32):
        return L.lce_preference_fwd_bwd(FAKE, FAKE, FAKE, FAKE, 1, None, 0.1, 0.0, 0, None, N, 64, 100, -100, chunk, 0, flags, FAKE,
                                        FAKE, FAKE, FAKE, FAKE, 1 << 40, None)
    for call in (policy, preference):
        assert call(N=9) == call(N=5, flags=32 | 16) == call(flags=32 | 1) == call(flags=32 | 8) == UNSUPPORTED
        assert call(flags=64) == INVALID
    assert L.lce_fwd_bwd_opt(FAKE, FAKE, FAKE, None, 4, 64, 100, -100, 4, 0, 32, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 40,
                             None) == INVALID
    n = ctypes.c_size_t(0)
    assert L.lce_workspace_size_opt(4, 64, 100, 4, 32, ctypes.byref(n)) == INVALID
    assert L.lce_policy_workspace_size(4, 64, 100, 4, 32, 1, ctypes.byref(n)) == 0


def test_policy_logits_arguments(L):
    for how in (dict(N=-1), dict(V=0), dict(ld=999), dict(dtype=3), dict(dtype=-1), dict(Z=None), dict(y=None), dict(ws=None),
                dict(loss=None), dict(red=3), dict(red=-1), dict(N=1 << 31), dict(V=(1 << 30) + 1, ld=1 << 31),
                dict(dZ=FAKE + 16), dict(dZ=FAKE + 6 * 1000)):   # dZ over a part of Z
        assert policy_logits(L, **how) == INVALID, how
    for how in (dict(Z=FAKE + 1), dict(Z=FAKE + 2, dtype=1), dict(y=FAKE + 4), dict(ws=FAKE + 8), dict(loss=FAKE + 2),
                dict(dloss=FAKE + 2), dict(dZ=FAR + 2), dict(Z=FAKE + 2)):
        assert policy_logits(L, **how) == ALIGN, how
    assert policy_logits(L, nbytes=2047) == WORKSPACE


def test_policy_head_arguments(L):
    def call(H=FAKE, W=FAKE, N=4, D=64, V=100, chunk=4, red=0, flags=0, loss=FAKE, dH=FAKE, dW=FAKE, ws=FAKE, nbytes=1 << 30):
        return L.lce_policy_fwd_bwd(H, W, FAKE, FAKE, None, None, None, 0.2, 0.2, 0.0, 1.0, None, N, D, V, -100, chunk, red,
                                    flags, loss, FAKE, dH, dW, ws, nbytes, None)
    for how in (dict(D=63), dict(N=-1), dict(V=0), dict(chunk=0), dict(H=None), dict(W=None), dict(dH=None), dict(dW=None),
                dict(ws=None), dict(loss=None), dict(flags=64), dict(flags=8 | 1), dict(red=5)):
        assert call(**how) == INVALID, how
    for how in (dict(H=FAKE + 8), dict(W=FAKE + 2), dict(dH=FAKE + 8), dict(dW=FAKE + 4), dict(ws=FAKE + 8), dict(loss=FAKE + 4)):
        assert call(**how) == ALIGN, how
    assert call(nbytes=100) == WORKSPACE
    assert call(flags=4) == UNSUPPORTED


def test_preference_arguments(L):
    def logits(Z=FAKE, dtype=0, ld=1000, y=FAKE, off=FAKE, pairs=3, ref=None, beta=0.1, e=0.0, dloss=None, N=9, V=1000, red=0,
               loss=FAKE, seq=FAKE, dZ=FAR, ws=FAKE, nbytes=1 << 20):
        return L.lce_preference_logits(Z, dtype, ld, y, off, pairs, ref, beta, e, 0, dloss, N, V, -100, red, loss, seq, dZ,
                                       ws, nbytes, None)

    def head(off=FAKE, pairs=3, ref=None, beta=0.1, e=0.0, dloss=None, N=9, D=64, V=100, chunk=4, red=0, flags=0, loss=FAKE,
             seq=FAKE, dH=FAKE, dW=FAKE, ws=FAKE, nbytes=1 << 30):
        return L.lce_preference_fwd_bwd(FAKE, FAKE, FAKE, off, pairs, ref, beta, e, 0, dloss, N, D, V, -100, chunk, red,
                                        flags, loss, seq, dH, dW, ws, nbytes, None)
    for how in (dict(off=None), dict(pairs=0), dict(pairs=-1), dict(beta=math.nan), dict(beta=math.inf), dict(e=-0.1), dict(e=1.1),
                dict(red=3), dict(loss=None), dict(seq=None), dict(N=-1), dict(ws=None)):
        assert logits(**how) == INVALID and head(**how) == INVALID, how
    for how in (dict(off=FAKE + 4), dict(ref=FAKE + 2), dict(dloss=FAKE + 1), dict(loss=FAKE + 2), dict(seq=FAKE + 2),
                dict(ws=FAKE + 8)):
        assert logits(**how) == ALIGN and head(**how) == ALIGN, how
    assert logits(nbytes=1024) == WORKSPACE and head(nbytes=1024) == WORKSPACE
    assert head(flags=4) == UNSUPPORTED
    for how in (dict(flags=64), dict(flags=9), dict(D=60), dict(chunk=0), dict(dH=None), dict(dW=None), dict(pairs=(1 << 24) + 1)):
        assert head(**how) == INVALID, how
    assert logits(dZ=FAKE + 64) == INVALID and logits(dZ=FAR + 4) == ALIGN
    n = ctypes.c_size_t(0)
    assert L.lce_preference_workspace_size(9, 64, 100, 4, 3, 0, 1, None) == INVALID
    assert L.lce_preference_workspace_size(9, 64, 100, 4, 0, 0, 1, ctypes.byref(n)) == INVALID
    assert L.lce_preference_logits_workspace_size(9, 0, ctypes.byref(n)) == INVALID
    sizes = []
    for grad, chunk, flags in ((0, 8, 0), (1, 8, 0), (1, 8, 16)):
        assert L.lce_preference_workspace_size(20, 64, 50000, chunk, 3, flags, grad, ctypes.byref(n)) == OK
        sizes.append(n.value)
    assert sizes[0] < sizes[2] < sizes[1]            # no chunk buffer; one; two


def test_scale_arguments(L):
    def scale(src=FAKE, s=1, g=FAKE, n=10, dst=FAR, d=1):
        return L.lce_scale(src, s, g, n, dst, d, None)
    for how in (dict(n=-1), dict(s=3), dict(d=-1), dict(g=None), dict(src=None), dict(dst=None), dict(dst=FAKE + 4),
                dict(dst=FAKE, d=0)):
        assert scale(**how) == INVALID, how
    for how in (dict(src=FAKE + 2), dict(dst=FAR + 2), dict(g=FAKE + 2)):
        assert scale(**how) == ALIGN, how


def test_int4_arguments(L):
    def quantize(W=FAKE, dtype=0, ldw=100, V=4, D=100, group=32, q=FAKE, ldq=64, s=FAKE, st=0, lds=4):
        return L.lce_int4_quantize(W, dtype, ldw, V, D, group, q, ldq, s, st, lds, None)

    def linear(X=FAKE, dtype=0, ldx=100, q=FAKE, ldq=64, s=FAKE, lds=4, group=32, M=9, V=4, D=100, out=FAKE, ldc=4, ws=FAKE,
               nbytes=1 << 20):
        return L.lce_int4_linear(X, dtype, ldx, q, ldq, s, lds, group, M, V, D, out, ldc, ws, nbytes, None)
    for how in (dict(dtype=3), dict(st=1), dict(group=48), dict(V=-1), dict(D=0), dict(D=65537, ldw=1 << 20, ldq=1 << 20, lds=4096),
                dict(ldw=99), dict(ldq=48), dict(lds=3), dict(W=None), dict(q=None), dict(s=None)):
        assert quantize(**how) == INVALID, how
    for how in (dict(ldq=72), dict(q=FAKE + 8), dict(W=FAKE + 1), dict(W=FAKE + 2, dtype=1), dict(s=FAKE + 1)):
        assert quantize(**how) == ALIGN, how
    for how in (dict(dtype=1), dict(group=16), dict(M=-1), dict(M=(1 << 20) + 1), dict(V=0), dict(D=0), dict(ldx=99), dict(ldc=3),
                dict(ldq=48), dict(lds=3), dict(X=None), dict(q=None), dict(s=None), dict(out=None), dict(ws=None)):
        assert linear(**how) == INVALID, how
    for how in (dict(ldq=72), dict(q=FAKE + 8), dict(X=FAKE + 1), dict(s=FAKE + 1), dict(out=FAKE + 1), dict(ws=FAKE + 8)):
        assert linear(**how) == ALIGN, how
    assert linear(nbytes=1024) == WORKSPACE
    n = ctypes.c_size_t(7)
    assert L.lce_int4_linear_workspace_size(1, 4096, 128, ctypes.byref(n)) == OK and n.value == 0
    assert L.lce_int4_linear_workspace_size(9, 100, 32, ctypes.byref(n)) == OK and n.value == 2048 + 9 * 256
    assert L.lce_int4_linear_workspace_size(9, 100, 33, ctypes.byref(n)) == INVALID


def test_python_calls_refuse_host_tensors():
    z, y, a, off = torch.randn(4, 8), torch.zeros(4, dtype=torch.int64), torch.zeros(4), torch.tensor([0, 2, 4])
    h, w = torch.randn(4, 8).bfloat16(), torch.randn(9, 8).bfloat16()
    for call in (lambda: lce.policy_logits(z, y, a), lambda: lce.policy_fwd_bwd(h, w, y, a), lambda: lce.policy_forward(h, w, y, a),
                 lambda: lce.linear_policy_loss(h, w, y, a), lambda: lce.preference_logits(z, y, off),
                 lambda: lce.preference_fwd_bwd(h, w, y, off), lambda: lce.linear_preference_loss(h, w, y, off),
                 lambda: lce.int4_weight(z), lambda: lce.int4_linear(h, lce.Int4Weight(z, z, 32))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: lce.linear_policy_loss(h, w, y, a, reduction="none"),
                 lambda: lce.linear_preference_loss(h, w, y, off, reduction="none")):
        with pytest.raises(ValueError, match="reduction"):
            call()


# ---------------------------------------------------------------- the oracle

def along(f, x, seed):
    """Difference of f along a direction u, and u."""
    u = np.random.default_rng(seed).standard_normal(x.shape)
    h = 1e-6
    return (f(x + h * u) - f(x - h * u)) / (2 * h), u


@pytest.mark.parametrize("reduction", ["mean", "sum"])
def test_oracle_policy_gradient_is_that_of_its_loss(reduction):
    g = np.random.default_rng(0)
    Z, y, a, w = g.standard_normal((12, 30)) * 2, g.integers(0, 30, 12), g.standard_normal(12), g.random(12)
    y[3] = -100
    logp = ao.log_softmax_of(Z, y, 0.7)[0]
    old, ref = logp + 0.3 * g.standard_normal(12), logp + 0.3 * g.standard_normal(12)
    kw = dict(old=old, ref=ref, weights=w, beta=0.2, temperature=0.7, reduction=reduction)
    d, u = along(lambda z: ao.policy(z, y, a, **kw)["loss"], Z, 1)
    assert abs(d - (ao.policy(Z, y, a, **kw)["dZ"] * u).sum()) <= 1e-7
    # from the definition, row by row
    p = np.exp(Z / 0.7) / np.exp(Z / 0.7).sum(1, keepdims=True)
    rows = 0.0
    for i in range(12):
        if y[i] >= 0:
            r = p[i, y[i]] / math.exp(old[i])
            q = math.exp(ref[i]) / p[i, y[i]]
            rows += w[i] * (-min(r * a[i], min(max(r, 0.8), 1.2) * a[i]) + 0.2 * (q - 1 - math.log(q)))
    assert abs(ao.policy(Z, y, a, **kw)["loss"] - rows / (11 if reduction == "mean" else 1)) <= 1e-12


@pytest.mark.parametrize("average,smoothing", [(False, 0.0), (True, 0.1)])
def test_oracle_preference_gradient_is_that_of_its_loss(average, smoothing):
    g = np.random.default_rng(2)
    Z, y, off = g.standard_normal((20, 15)), g.integers(0, 15, 20), np.array([1, 4, 4, 11, 18])
    y[[2, 7]] = -100
    ref = g.standard_normal(4)
    d, u = along(lambda z: ao.preference(z, y, off, ref, 0.5, smoothing, average)["loss"], Z, 3)
    o = ao.preference(Z, y, off, ref, 0.5, smoothing, average)
    assert abs(d - (o["dZ"] * u).sum()) <= 1e-8
    assert not o["dZ"][[0, 2, 7, 18, 19]].any()
    lp = np.log(np.exp(Z) / np.exp(Z).sum(1, keepdims=True))[np.arange(20), np.maximum(y, 0)] * (y >= 0)
    seq = [lp[a:b].sum() / (max(1, (y[a:b] >= 0).sum()) if average else 1) for a, b in zip(off, off[1:])]
    loss = 0.0
    for k in range(2):
        m = 0.5 * ((seq[k] - ref[k]) - (seq[2 + k] - ref[2 + k]))
        s = 1 / (1 + math.exp(-m))
        loss -= ((1 - smoothing) * math.log(s) + smoothing * math.log(1 - s)) / 2
    assert abs(o["loss"] - loss) <= 1e-12


def test_oracle_int4_packs_what_it_unpacks():
    g = np.random.default_rng(4)
    W = g.standard_normal((5, 70)) * 0.1
    q, s = ao.quantize_int4(W, 32, lambda x: x.astype(np.float16).astype(np.float64))
    packed = np.full((5, 35), 0, np.uint8)
    packed[:] = (q[:, 0::2] + 8).astype(np.uint8) | ((q[:, 1::2] + 8).astype(np.uint8) << 4)
    full = ao.int4_values(packed, s, 32, 70)
    step = np.repeat(s, 32, 1)[:, :70]
    assert np.allclose(full, q * step) and (np.abs(full - W) <= 0.5001 * step).all()
