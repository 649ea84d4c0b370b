"""4-bit linear layers at the ends of their range: weights beyond the scale's type, and a wait that runs out."""
import math

import numpy as np
import pytest
import torch

import linear_cross_entropy_chunked_gb300 as lce
from linear_cross_entropy_chunked_gb300 import _binding as _b
from oracle import answers_oracle as ao
from tests.test_gpu_int4 import check, values, weight

pytestmark = pytest.mark.gpu

TIMEOUT = 5


@pytest.mark.parametrize("m,v,d,group", [(9, 130, 96, 32), (7, 300, 4096, 128), (100, 25700, 512, 64), (300, 1001, 8192, 32)])
def test_a_wait_that_runs_out_leaves_nan(m, v, d, group):
    # no stage of the weight comes, as if its copies were lost: every result is NaN, in all tiles of every CTA, for a
    # caller who reads no status too
    g = torch.Generator().manual_seed(m)
    X = torch.randn(m, d, generator=g).bfloat16().cuda()
    w = weight(v, d, group, torch.bfloat16, m)
    out = torch.ones(m, v + 5, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(lce.int4_workspace_size(m, d, group), dtype=torch.uint8, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    status = _b.lib().lce_selftest_int4_timeout(
        X.data_ptr(), 0, d, w.q.data_ptr(), w.q.stride(0), w.scale.data_ptr(), w.scale.stride(0), group, m, v, d,
        out.data_ptr(), v + 5, ws.data_ptr(), ws.numel(), 1000, s)
    assert status == 0
    assert lce.read_status(ws) == TIMEOUT and lce.read_status(ws) == 0
    assert torch.isnan(out[:, :v]).all() and (out[:, v:] == 1).all()
    lce.int4_linear(X, w, out=out[:, :v], ws=ws)
    assert lce.read_status(ws) == 0
    check(out[:, :v], X, values(w, d))
    assert math.isfinite(out.float().sum().item())


@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("wtype", [torch.float32, torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("stype", [torch.float16, torch.bfloat16], ids=str)
def test_groups_beyond_the_range_of_their_scale(stype, wtype, group):
    # groups whose largest magnitude goes from the type's smallest number to its largest, each number a whole multiple
    # (-7 .. 7) of a seventh of it where the types have that, and a group of zeros
    lo, hi = {torch.float32: (-149, 128), torch.bfloat16: (-133, 128), torch.float16: (-24, 16)}[wtype]
    g = torch.Generator().manual_seed(group)
    top = torch.tensor([2.0 ** e * 1.25 for e in range(lo, hi)] + [0.0], dtype=torch.float64)
    top = top.clamp(max=torch.finfo(wtype).max)
    whole = torch.randint(-7, 8, (len(top), group), generator=g).double()
    whole[:, 3] = 7
    W = (whole / 7 * top[:, None]).to(wtype)
    w = lce.int4_weight(W.cuda(), group, stype)
    x = W.double().numpy()
    big = np.abs(x).max(1)
    small, largest = {torch.float16: (2.0 ** -24, 65504.0), torch.bfloat16: (2.0 ** -133, torch.finfo(stype).max)}[stype]
    want = np.where(big > 0, np.clip(big / 7, small, largest), 1.0)
    scale = w.scale.double().cpu().numpy()[:, 0]
    # one rounding to the type (a seventh in fp32 first), or half of its smallest step, which is its smallest number
    half = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}[stype]
    assert (scale > 0).all() and (np.abs(scale - want) <= np.maximum((half + 2.0 ** -23) * want, small * 0.501)).all()
    assert (scale[big == 0] == 1).all()
    # the nearest value of -8 .. 7, up to the quotient's rounding in fp32
    q = ao.int4_values(w.q.cpu().numpy(), np.ones_like(scale)[:, None], group, group)
    near = np.clip(x / scale[:, None], -8, 7)
    assert (np.abs(q - near) <= 0.5 + 1e-5).all()
    lost = big > 14 * small    # (what the scale can tell from nothing)
    assert (np.abs(q).max(1)[lost] > 0).all()
