"""Attention's limits of rows: the kernels round row numbers up to whole tiles in 32 bits.
Each call returns before any CUDA call (the pointers are never used), so this runs without
a GPU."""
import pytest

from test_paged_refusals import L, w  # noqa: F401  (fixtures)
from test_operators_abi import attention
from test_paged_refusals import paged

INVALID, SHAPE = 1, 3
MOST = (1 << 31) - 1025  # rows of Q times heads of a group
NOWHERE = dict(O=None)   # refused after the shapes have been looked at


@pytest.mark.parametrize("hq,hk", [(1, 1), (4, 4), (4, 2), (12, 1)])
def test_paged_attention(L, hq, hk):  # noqa: F811
    most = MOST // (hq // hk)
    for tq in (most + 1, (1 << 31) // (hq // hk) - 1):
        assert paged(L, Tq=tq, Hq=hq, Hk=hk, **NOWHERE) == SHAPE, tq
    assert paged(L, Tq=most, Hq=hq, Hk=hk, **NOWHERE) == INVALID


@pytest.mark.parametrize("hq,hk", [(1, 1), (4, 4), (4, 2), (12, 1)])
def test_attention(L, hq, hk):  # noqa: F811
    most = MOST // (hq // hk)
    for tq in (most + 1, (1 << 31) // (hq // hk) - 1):
        assert attention(L, Tq=tq, Hq=hq, Hk=hk, **NOWHERE) == SHAPE, tq
    assert attention(L, Tq=most, Hq=hq, Hk=hk, **NOWHERE) == INVALID
    for tk in (MOST + 1, (1 << 31) - 1):
        assert attention(L, Tk=tk, Hq=hq, Hk=hk, **NOWHERE) == SHAPE, tk
    assert attention(L, Tk=MOST, Hq=hq, Hk=hk, **NOWHERE) == INVALID
