"""The device status of the products inside fp8_linear. A wait that runs out is stood in for: after the product in
question the library's self-test (a bounded wait that nothing ends) leaves its status in the same workspace."""
import pytest
import torch

import linear_cross_entropy_chunked_gb300 as lce
from linear_cross_entropy_chunked_gb300 import _binding

pytestmark = pytest.mark.gpu
OK, TIMEOUT = 0, 5


class Library:
    """The library, whose product number `late` of those counted from here ends by a timeout."""

    def __init__(self, late):
        self._lib, self._late, self.products = _binding.lib(), late, 0

    def __getattr__(self, name):
        call = getattr(self._lib, name)
        if name not in ("lce_fp8_matmul", "lce_fp8_linear"):
            return call

        def product(*args):
            st = call(*args)
            if self.products == self._late:
                assert self._lib.lce_selftest_wait_timeout(args[-3], 1024, 1000, args[-1]) == OK
            self.products += 1
            return st
        return product


def inputs(m=40, v=300, d=136):
    g = torch.Generator().manual_seed(1)
    X, W, dZ = (torch.randn(*s, generator=g).bfloat16().cuda() for s in ((m, d), (v, d), (m, v)))
    return X.requires_grad_(), W.requires_grad_(), dZ, torch.zeros(1024, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("late,products", [(None, 3), (0, 3), (1, 3), (2, 3)])
def test_training(monkeypatch, late, products):
    X, W, dZ, status = inputs()
    want = lce.fp8_linear(X, W)
    want = (want.detach(), *torch.autograd.grad(want, (X, W), dZ))
    fake = Library(late)
    monkeypatch.setattr(_binding, "lib", lambda: fake)
    Z = lce.fp8_linear(X, W, status=status)
    got = (Z.detach(), *torch.autograd.grad(Z, (X, W), dZ))
    assert fake.products == products and all(torch.equal(a, b) for a, b in zip(got, want))
    assert lce.read_status(status) == (OK if late is None else TIMEOUT)
    assert lce.read_status(status) == OK       # cleared


@pytest.mark.parametrize("late", [None, 0, 1])
def test_frozen(monkeypatch, late):
    X, W, dZ, status = inputs()
    w8 = lce.fp8_weight(W.detach())
    fake = Library(late)
    monkeypatch.setattr(_binding, "lib", lambda: fake)
    torch.autograd.grad(lce.fp8_linear(X, w8, status=status), X, dZ)
    assert fake.products == 2 and lce.read_status(status) == (OK if late is None else TIMEOUT)
    fake = Library(0)
    with torch.no_grad():
        lce.fp8_linear(X, w8, status=status)
    assert fake.products == 1 and lce.read_status(status) == TIMEOUT


def test_one_status_for_several_layers_and_a_graph():
    X, W, dZ, status = inputs()
    w8 = lce.fp8_weight(W.detach())
    with torch.no_grad():
        want = lce.fp8_linear(X, w8, status=status)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            Z = lce.fp8_linear(X, w8, status=status)
    graph.replay()
    assert torch.equal(Z, want) and lce.read_status(status) == OK
    lce.selftest_wait_timeout(status, 1000)    # an earlier product's
    graph.replay()
    assert lce.read_status(status) == TIMEOUT  # stays until it is read


def test_refusals():
    X, W, _, status = inputs()
    for bad in (status[:1000], status.float(), status.cpu(), torch.zeros(2048, dtype=torch.uint8, device="cuda")[::2],
                torch.zeros(1040, dtype=torch.uint8, device="cuda")[1:1025]):
        with pytest.raises(ValueError):
            lce.fp8_linear(X, W, status=bad)
