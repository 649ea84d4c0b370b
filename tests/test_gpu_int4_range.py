"""4-bit linear layers where a wait runs out."""
import math

import pytest
import torch

import linear_cross_entropy_chunked_gb300 as lce
from linear_cross_entropy_chunked_gb300 import _binding as _b
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
