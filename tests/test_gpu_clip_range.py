"""The 2-norm of finite values whose squares, or sums of squares, do not fit fp32, and clipping by it.

The tolerances of the ordinary range: a thread's squares round as there or (in fp64) less, so the norm is
within 19 * 2^-24 of the oracle's, the factor within 3 roundings more. A factor below fp32's normal numbers
is a multiple of 2^-149: off by half of that besides."""
import math

import numpy as np
import pytest
import torch

import linear_cross_entropy_chunked_gb300 as lce
from oracle import ops_oracle

pytestmark = pytest.mark.gpu

NORM_REL = 19 * 2.0 ** -24
FACTOR_REL = NORM_REL + 3 * 2.0 ** -24


def check(host, max_norm, norm_type=2.0):
    dev = [h.cuda() for h in host]
    want, scaled = ops_oracle.clip([h.double().numpy() for h in host], max_norm, norm_type)
    norm = lce.grad_norm(dev, norm_type)
    assert abs(norm.item() - want) <= NORM_REL * want + 2.0 ** -150, (norm.item(), want)
    assert lce.clip_grad_norm(dev, max_norm, norm_type=norm_type).item() == norm.item()
    factor = min(1.0, max_norm / (want + 1e-6))
    rel = FACTOR_REL + (2.0 ** -150 / factor if factor < 2.0 ** -126 else 0.0)
    for h, w, d in zip(host, scaled, dev):
        t = torch.finfo(h.dtype)
        err = np.abs(d.double().cpu().numpy() - w)
        assert (err <= (t.eps / 2 + rel) * np.abs(w) + t.smallest_normal * t.eps / 2).all()


def values(n, scale, dtype, seed=0):
    g = torch.Generator().manual_seed(seed + n)
    return (torch.randn(n, generator=g).double() * scale).to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [1, 16, 33, 5000, 2_000_003])
@pytest.mark.parametrize("scale", [1e34, 1e30, 1e19, 5e18, 1e18, 3e17, 1e15, 1.0, 1e-15, 1e-18, 1e-20, 1e-23, 1e-25, 1e-30,
                                   1e-37, 1e-40])
def test_range_of_the_2_norm(scale, n, dtype):
    check([values(n, scale, dtype)], 1.0 if scale > 1 else 0.25 * scale)


@pytest.mark.parametrize("scale", [1e34, 1e18, 1e-20, 1e-30])
def test_thousands_of_chunks_per_thread(scale):
    # one sum that grows over many chunks; 2^28 equal values
    g = torch.full((1 << 28,), scale, device="cuda")
    want = float(np.float32(scale)) * 2.0 ** 14
    assert abs(lce.grad_norm(g).item() - want) <= NORM_REL * want


def test_values_of_all_sizes_at_once():
    mixed = torch.cat([values(1000, s, torch.float32) for s in (1e18, 1.0, 1e-30, 0.0, 1e10, 1e-12)])
    check([mixed[torch.randperm(6000, generator=torch.Generator().manual_seed(1))]], 1.0)
    check([values(4000, 1e18, torch.float32), values(3000, 1e-3, torch.float16), values(5, 1e-30, torch.bfloat16)], 1.0)
    check([values(4000, 1e-30, torch.float32), torch.zeros(100_000), values(70, 1e-27, torch.bfloat16)], 1e-30)
    check([values(60_000, 1e-9, torch.float16)], 1e-7)          # subnormal halves
    # one large value in a tensor, at its ends and inside
    for at in (0, 7, 4096, 49_999):
        x = values(50_000, 1.0, torch.float32)
        x[at] = -3e38
        check([x], 1.0)


@pytest.mark.parametrize("kind", [2.0, 1.0, math.inf])
def test_beyond_fp32(kind):
    # the norm itself does not fit: infinite, and the factor 0
    g = torch.full((100_000,), 3e38, device="cuda")
    assert lce.clip_grad_norm(g, 1.0, norm_type=kind).item() == (math.inf if kind != math.inf else float(np.float32(3e38)))
    assert (g == 0).all() if kind != math.inf else (g > 0).all()


def test_signed_zeros_and_offsets():
    for off in (0, 1, 3):
        x = torch.zeros(70_001 + off, device="cuda", dtype=torch.bfloat16)[off:]
        x[::2] = -0.0
        assert lce.grad_norm(x).item() == 0.0
        x[1234] = 1e-30
        assert lce.grad_norm(x).item() == pytest.approx(float(torch.tensor(1e-30).bfloat16()), rel=NORM_REL)
