"""What the weight gradient of a loss on answers is kept in until the upstream gradient is known."""
import pytest
import torch

import linear_cross_entropy_chunked_gb300 as lce

pytestmark = pytest.mark.gpu


def inputs(n, d, v, seed):
    g = torch.Generator().manual_seed(seed)
    H = torch.randn(n, d, generator=g).bfloat16().cuda().requires_grad_()
    W = (torch.randn(v, d, generator=g) / 8).bfloat16().cuda().requires_grad_()
    return H, W, torch.randint(0, v, (n,), generator=g).cuda(), torch.randn(n, generator=g).cuda()


@pytest.mark.parametrize("which", ["policy", "preference"])
@pytest.mark.parametrize("dtype", [None, torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("upstream", [1.0, 1 / 3, 0.25, 0.0])
def test_roundings_of_the_weight_gradient(which, dtype, upstream):
    H, W, y, a = inputs(300, 64, 500, 1)
    off = torch.tensor([0, 80, 150, 220, 300], device="cuda")
    if which == "policy":
        loss = lce.linear_policy_loss(H, W, y, a, dW_dtype=dtype)[0]
        dW = lce.policy_fwd_bwd(H.detach(), W.detach(), y, a)[3]
    else:
        loss = lce.linear_preference_loss(H, W, y, off, dW_dtype=dtype)[0]
        dW = lce.preference_fwd_bwd(H.detach(), W.detach(), y, off)[3]
    loss.backward(torch.tensor(upstream, device="cuda"))
    # fp32 sums, scaled in fp32, then rounded: once, or before too
    first = dW if dtype == torch.float32 else dW.bfloat16().float()
    scaled = first * torch.tensor(upstream, device="cuda")
    assert W.grad.dtype == torch.bfloat16 and torch.equal(W.grad, scaled.bfloat16())
    if dtype == torch.float32:
        exact = dW.double() * upstream
        # half a step of bf16 (numbers from 1 to 2 are 2^-7 apart), and fp32's of the product
        assert ((W.grad.double() - exact).abs() <= (2.0 ** -8 + 2.0 ** -23) * exact.abs() + 2.0 ** -134).all()


def test_what_is_refused():
    H, W, y, a = inputs(300, 64, 500, 2)
    off = torch.tensor([0, 80, 150, 220, 300], device="cuda")
    for call, args in ((lce.linear_policy_loss, (H, W, y, a)), (lce.linear_preference_loss, (H, W, y, off))):
        with pytest.raises(TypeError):
            call(*args, dW_dtype=torch.float16)
        with pytest.raises(ValueError):
            call(*args, dW_dtype=torch.bfloat16, chunk=149)
        with pytest.raises(ValueError):
            call(*args, dW_dtype=torch.bfloat16, chunk=299, low_memory=True)
        call(*args, dW_dtype=torch.bfloat16, chunk=150)[0].backward()
        call(*args, dW_dtype=torch.float32, chunk=64)[0].backward()
