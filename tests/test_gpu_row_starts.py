"""16-bit rows at every address: the kernels read words, but only such as lie inside a row. A row's neighbours,
up to the ends of its memory, hold NaN and infinities in turn, and no bit of a result depends on them."""
import numpy as np
import pytest
import torch

import linear_cross_entropy_chunked_gb300 as lce
from oracle import ops_oracle

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def views(x, fill):
    """x [R, C] at every offset of 16 bytes, alone in its memory or among `fill`."""
    r, c = x.shape
    for at in range(8):
        for gap in (0, 1, 2, 7):
            flat = torch.full((at + r * (c + gap) + 8,), fill, dtype=x.dtype, device="cuda")
            v = flat[at:at + r * (c + gap)].view(r, c + gap)[:, :c]
            v.copy_(x)
            yield v


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("c", [8, 9, 15, 16, 136, 257, 1001])
def test_sampling(c, dtype):
    g = torch.Generator().manual_seed(c)
    z = (torch.randn(5, c, generator=g) * 2).to(DTYPES[dtype])
    z[0, 0] = z[1, -1] = 9.0                   # the ends matter
    u = torch.rand(5, generator=g)
    ref = ops_oracle.sample(z.double().numpy(), u.double().numpy(), 1.0, 0, 0.95, 0.0)
    for fill in (float("nan"), float("inf")):
        for v in views(z, fill):
            tokens, _ = lce.sample_logits(v, u.cuda(), top_p=0.95)
            np.testing.assert_array_equal(tokens.cpu().numpy(), ref["tokens"])
            assert torch.equal(lce.sample_logits(v, u.cuda(), temperature=0.0)[0].cpu(), z.float().argmax(1))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("c", [8, 9, 16, 121, 128, 136, 257])
def test_quantisation(c, dtype):
    x = torch.randn(3, c, generator=torch.Generator().manual_seed(c)).to(DTYPES[dtype])
    want = [ops_oracle.quantize_fp8(m, t) for m, t in ((x.double().numpy(), False), (x.double().numpy(), True),
                                                       (x.double().numpy().T, False))]
    for fill in (float("nan"), float("inf")):
        for v in views(x, fill):
            for (q, s), (wq, ws) in zip((lce.quantize_fp8(v), lce.quantize_fp8(v, tiles=True),
                                         lce.quantize_fp8(v, transpose=True)), want):
                np.testing.assert_array_equal(s.double().cpu().numpy(), ws)
                np.testing.assert_array_equal(q.float().double().cpu().numpy(), wq)
