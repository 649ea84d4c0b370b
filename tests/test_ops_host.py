"""Host-side tests of sampling, the 8-bit linear layer and gradient clipping (no GPU): argument errors of the
C ABI, refusals of the Python calls, and the fp64 oracle against independent definitions. Pointer
arguments are fake addresses that the library must reject before it touches the device."""
import ctypes
import itertools
import math

import numpy as np
import pytest
import torch

import linear_cross_entropy_chunked_gb300 as lce
from oracle import ops_oracle

OK, INVALID, ALIGN, WORKSPACE = 0, 1, 2, 3
FAKE = 0x10000000


@pytest.fixture(scope="module")
def L():
    try:
        lce.build()
    except RuntimeError as e:  # no nvcc here
        pytest.skip(str(e))
    return lce.lib()


def sample(L, Z=FAKE, dtype=0, ld=1000, N=4, V=1000, u=FAKE, t=None, k=None, tokens=FAKE, logprobs=FAKE):
    return L.lce_sample_logits(Z, dtype, ld, N, V, u, t, k, None, None, 1.0, 0, 1.0, 0.0, tokens, logprobs, None)


def test_sample_arguments(L):
    assert sample(L, N=-1) == INVALID
    assert sample(L, V=0) == INVALID
    assert sample(L, V=(1 << 20) + 1, ld=1 << 21) == INVALID
    assert sample(L, ld=999) == INVALID
    assert sample(L, dtype=3) == INVALID
    assert sample(L, dtype=-1) == INVALID
    assert sample(L, Z=None) == INVALID
    assert sample(L, u=None) == INVALID
    assert sample(L, tokens=None) == INVALID
    assert sample(L, N=(1 << 27) + 1) == INVALID
    assert sample(L, Z=FAKE + 1) == ALIGN
    assert sample(L, Z=FAKE + 2, dtype=1) == ALIGN
    assert sample(L, u=FAKE + 2) == ALIGN
    assert sample(L, tokens=FAKE + 4) == ALIGN
    assert sample(L, logprobs=FAKE + 1) == ALIGN
    assert sample(L, t=FAKE + 2) == ALIGN


def quantize(L, X=FAKE, dtype=0, ld=256, R=10, C=256, q=FAKE, ldq=256, s=FAKE, qt=None, ldqt=0, st=None):
    return L.lce_fp8_quantize(X, dtype, ld, R, C, 0, q, ldq, s, qt, ldqt, st, None)


def test_quantize_arguments(L):
    assert quantize(L, R=-1) == INVALID
    assert quantize(L, C=0) == INVALID
    assert quantize(L, ld=255) == INVALID
    assert quantize(L, dtype=7) == INVALID
    assert quantize(L, q=None) == INVALID              # nothing to write
    assert quantize(L, s=None) == INVALID
    assert quantize(L, ldq=240) == INVALID
    assert quantize(L, qt=FAKE, ldqt=16, st=None) == INVALID
    assert quantize(L, qt=FAKE, ldqt=0, st=FAKE) == INVALID
    assert quantize(L, X=None) == INVALID
    assert quantize(L, X=FAKE + 1) == ALIGN
    assert quantize(L, q=FAKE + 8) == ALIGN
    assert quantize(L, ldq=264) == ALIGN
    assert quantize(L, qt=FAKE, ldqt=24, st=FAKE) == ALIGN
    assert quantize(L, s=FAKE + 2) == ALIGN


def matmul(L, A=FAKE, lda=512, sa=FAKE, B=FAKE, ldb=512, sb=FAKE, M=8, N=64, K=512, out=FAKE, ldc=64, dtype=0,
           ws=FAKE, ws_bytes=1024, strides=(4, 1, 4, 1)):
    return L.lce_fp8_matmul(A, lda, sa, strides[0], strides[1], B, ldb, sb, strides[2], strides[3], 0, M, N, K, out,
                            ldc, dtype, ws, ws_bytes, None)


def test_matmul_arguments(L):
    assert matmul(L, M=-1) == INVALID
    assert matmul(L, N=-1) == INVALID
    assert matmul(L, K=0) == INVALID
    assert matmul(L, lda=496) == INVALID
    assert matmul(L, ldb=496) == INVALID
    assert matmul(L, ldc=56) == INVALID
    assert matmul(L, dtype=3) == INVALID
    assert matmul(L, strides=(4, -1, 4, 1)) == INVALID
    for name in ("A", "sa", "B", "sb", "out", "ws"):
        assert matmul(L, **{name: None}) == INVALID, name
    for name in ("A", "B", "out", "ws"):
        assert matmul(L, **{name: FAKE + 8}) == ALIGN, name
    assert matmul(L, sa=FAKE + 2) == ALIGN
    assert matmul(L, lda=520) == ALIGN
    assert matmul(L, ldb=520) == ALIGN
    assert matmul(L, ldc=68) == ALIGN                  # bf16: 136 bytes
    assert matmul(L, ws_bytes=1023) == WORKSPACE
    n = ctypes.c_size_t(0)
    assert L.lce_fp8_matmul_workspace_size(ctypes.byref(n)) == OK and n.value == 1024
    assert L.lce_fp8_matmul_workspace_size(None) == INVALID


def test_fp8_linear_arguments(L):
    n = ctypes.c_size_t(0)
    assert L.lce_fp8_linear_workspace_size(5, 300, ctypes.byref(n)) == OK
    assert n.value == 1024 + 1024 + 5 * 304
    assert L.lce_fp8_linear_workspace_size(-1, 300, ctypes.byref(n)) == INVALID
    assert L.lce_fp8_linear_workspace_size(5, 0, ctypes.byref(n)) == INVALID

    def linear(X=FAKE, dtype=0, W=FAKE, ldw=304, sw=FAKE, out=FAKE, ldc=64, ws=FAKE, ws_bytes=1 << 20, ldx=300):
        return L.lce_fp8_linear(X, dtype, ldx, W, ldw, sw, 3, 1, 5, 64, 300, out, ldc, 0, ws, ws_bytes, None)
    assert linear(ws=None) == INVALID
    assert linear(ws_bytes=n.value - 1) == WORKSPACE
    assert linear(ws=FAKE + 8) == ALIGN
    assert linear(W=None) == INVALID
    assert linear(W=FAKE + 8) == ALIGN
    assert linear(ldw=300) == ALIGN
    assert linear(out=FAKE + 2) == ALIGN
    assert linear(X=None) == INVALID
    assert linear(dtype=5) == INVALID
    assert linear(ldx=299) == INVALID


def clip(L, ptrs=(FAKE, FAKE + 4096), sizes=(1000, 10), dtypes=(0, 1), outs=None, kind=0, max_norm=1.0, eps=1e-6,
         norm=FAKE + (1 << 20), ws=FAKE + (2 << 20), ws_bytes=1 << 20, n=None):
    k = len(ptrs)
    arr = (ctypes.c_void_p * k)(*ptrs)
    out = None if outs is None else (ctypes.c_void_p * k)(*outs)
    return L.lce_clip_grad_norm(arr, (ctypes.c_int64 * k)(*sizes), (ctypes.c_int32 * k)(*dtypes), out,
                                k if n is None else n, kind, max_norm, eps, norm, ws, ws_bytes, None)


def test_clip_arguments(L):
    assert clip(L, n=-1) == INVALID
    assert clip(L, kind=3) == INVALID
    assert clip(L, max_norm=-1.0) == INVALID
    assert clip(L, max_norm=math.nan) == INVALID
    assert clip(L, eps=-1.0) == INVALID
    assert clip(L, dtypes=(0, 5)) == INVALID
    assert clip(L, sizes=(1000, -1)) == INVALID
    assert clip(L, ptrs=(FAKE, None)) == INVALID
    assert clip(L, norm=None) == INVALID
    assert clip(L, ws=None) == INVALID
    assert clip(L, ptrs=(FAKE + 1, FAKE + 4096)) == ALIGN
    assert clip(L, ptrs=(FAKE, FAKE + 4098)) == ALIGN   # fp32
    assert clip(L, ws=FAKE + 8) == ALIGN
    assert clip(L, ws_bytes=8 * 1024 - 1) == WORKSPACE
    n = ctypes.c_size_t(0)
    assert L.lce_grad_norm_workspace_size(1024, ctypes.byref(n)) == OK and n.value == 8192
    assert L.lce_grad_norm_workspace_size(1025, ctypes.byref(n)) == OK and n.value == 2 * 8192
    assert L.lce_grad_norm_workspace_size(0, ctypes.byref(n)) == OK and n.value == 8192
    assert L.lce_grad_norm_workspace_size(-1, ctypes.byref(n)) == INVALID


def test_clip_refuses_overlaps(L):
    # 1000 bf16 values are 2000 bytes
    assert clip(L, ptrs=(FAKE, FAKE), dtypes=(0, 0)) == INVALID                  # the same tensor twice
    assert clip(L, ptrs=(FAKE, FAKE + 1996), dtypes=(0, 1)) == INVALID           # its last values
    assert clip(L, ptrs=(FAKE + 1996, FAKE), sizes=(10, 1000), dtypes=(1, 0)) == INVALID
    # an output over another gradient, over part of its own, over another output
    assert clip(L, outs=(FAKE + 8192, FAKE)) == INVALID
    assert clip(L, outs=(FAKE + 2, FAKE + 4096), dtypes=(0, 1)) == INVALID
    assert clip(L, outs=(FAKE + 8192, FAKE + 8192 + 1996)) == INVALID


def test_python_calls_refuse_host_tensors():
    Z, u = torch.randn(2, 8), torch.rand(2)
    for call in (lambda: lce.sample_logits(Z, u), lambda: lce.grad_norm([Z]), lambda: lce.clip_grad_norm(Z, 1.0),
                 lambda: lce.quantize_fp8(Z), lambda: lce.fp8_weight(Z), lambda: lce.fp8_linear(Z, Z),
                 lambda: lce.fp8_matmul(Z, Z, Z, Z)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError):
        lce.clip_grad_norm([], 1.0)
    with pytest.raises(ValueError):
        lce.clip_grad_norm([Z], -1.0)
    with pytest.raises(ValueError):
        lce.grad_norm([Z], norm_type=3)


# ---------------------------------------------------------------- the oracle

def test_oracle_e4m3_is_the_format():
    bits = np.arange(1 << 16, dtype=np.uint16)
    x = torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16)
    x = x[torch.isfinite(x) & (x.abs() <= 448)]
    want = x.float().to(torch.float8_e4m3fn).float().double().numpy()
    np.testing.assert_array_equal(ops_oracle.e4m3(x.double().numpy()), want)


@pytest.mark.parametrize("tiles", [False, True])
def test_oracle_scales(tiles):
    g = np.random.default_rng(0)
    X = g.standard_normal((130, 300)) * 10.0 ** g.integers(-12, 12, (130, 1))
    X[5] = 0
    q, s = ops_oracle.quantize_fp8(X, tiles)
    assert np.abs(q).max() <= 448
    full = ops_oracle.dequantize_fp8(q, s)
    rows = np.repeat(s, 128, 0)[:130] if tiles else s
    step = np.repeat(rows, 128, 1)[:, :300] * 2.0 ** -9
    assert (np.abs(full - X) <= np.maximum(np.abs(X) * 2.0 ** -4, step / 2)).all()
    # half the scale would not do, unless the block is zero
    P = np.zeros((256 if tiles else 130, 384))
    P[:130, :300] = np.abs(X)
    amax = P.reshape(-1, 128 if tiles else 1, 3, 128).max(axis=(1, 3))
    assert ((amax > 448 * s / 2) | (amax == 0)).all() and (amax <= 448 * s).all()


def brute(z, u, T, k, p, q):
    """One row, by sorting explicit (logit, index) pairs."""
    order = sorted(range(len(z)), key=lambda i: (-z[i], i))
    w = {i: math.exp((z[i] - z[order[0]]) / T) for i in order}
    kept = order[:k] if k else order
    total, before, out = sum(w[i] for i in kept), 0.0, []
    for i in kept:
        if (not out or p >= 1 or before < p * total) and (not out or w[i] >= q):
            out.append(i)
        before += w[i]
    total, c = sum(w[i] for i in out), 0.0
    for i in sorted(out):
        c += w[i]
        if c > u * total:
            return i, math.log(w[i] / total)


def test_oracle_sampling():
    g = np.random.default_rng(1)
    for T, k, p, q in itertools.product((0.5, 1.0, 2.0), (0, 1, 5), (1.0, 0.75), (0.0, 0.125)):
        z = np.round(g.standard_normal((6, 20)) * 2, 1)
        u = g.random(6).astype(np.float32)
        r = ops_oracle.sample(z, u, T, k, p, q)
        for i in range(6):
            token, logp = brute(list(z[i]), float(u[i]), T, k, p, q)
            assert r["tokens"][i] == token and abs(r["logprobs"][i] - logp) < 1e-12


def test_oracle_clip():
    g = torch.Generator().manual_seed(3)
    grads = [torch.randn(n, generator=g, dtype=torch.float64) for n in (5, 100, 1)]
    for kind in (1.0, 2.0, math.inf):
        params = [torch.nn.Parameter(x.clone()) for x in grads]
        for p in params:
            p.grad = p.detach().clone()
        want = torch.nn.utils.clip_grad_norm_(params, 0.7, norm_type=kind)
        norm, scaled = ops_oracle.clip([x.numpy() for x in grads], 0.7, kind)
        assert abs(norm - want.item()) < 1e-12
        for p, s in zip(params, scaled):
            np.testing.assert_allclose(p.grad.numpy(), s, rtol=1e-12)


def test_matmul_best_workspace_arguments(L):
    n = ctypes.c_size_t(0)
    size = L.lce_fp8_matmul_best_workspace_size
    assert size(5, 5, 300, 0, None) == INVALID
    assert size(-1, 5, 300, 0, ctypes.byref(n)) == INVALID
    assert size(5, -1, 300, 0, ctypes.byref(n)) == INVALID
    assert size(5, 5, 0, 0, ctypes.byref(n)) == INVALID
    assert size(5, (1 << 30) + 1, 300, 0, ctypes.byref(n)) == INVALID
