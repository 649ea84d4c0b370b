"""Refusals of the 4-bit layer's self-test, without a GPU."""
import pytest

from tests.test_answers_host import ALIGN, FAKE, INVALID, L, WORKSPACE  # noqa: F401 (L is the fixture)


def selftest(L, X=FAKE, M=9, ws=FAKE, nbytes=1 << 20, limit=1000, group=32):
    return L.lce_selftest_int4_timeout(X, 0, 100, FAKE, 64, FAKE, 4, group, M, 4, 100, FAKE, 4, ws, nbytes, limit, None)


@pytest.mark.parametrize("how,want", [(dict(limit=0), INVALID), (dict(limit=2000001), INVALID), (dict(M=1), INVALID),
                                      (dict(M=0), INVALID), (dict(group=16), INVALID), (dict(X=None), INVALID),
                                      (dict(ws=None), INVALID), (dict(X=FAKE + 1), ALIGN), (dict(nbytes=1024), WORKSPACE)],
                         ids=str)
def test_selftest_arguments(L, how, want):  # noqa: F811
    assert selftest(L, **how) == want
