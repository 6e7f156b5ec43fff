"""Refusals of the rotary entry point for caches in pages: each returns before any CUDA call,
so this runs without a GPU."""
import pytest

from test_paged_refusals import APPEND, FAKE, ODD, OK, INVALID, ALIGN, SHAPE, L, w  # noqa: F401


def append(L, Q=FAKE, K=FAKE, V=FAKE, Qo=FAKE, Kc=FAKE, Vc=FAKE, dtype=0, T=4, Hq=4, Hk=2, D=64, rot=32, rows=160,
           page_size=16, strides=APPEND, pos=FAKE, slots=FAKE, freqs=FAKE, amp=1.0, layout=0):
    return L.w8a8_rotary_append_pages(Q, K, V, Qo, Kc, Vc, dtype, T, Hq, Hk, D, rot, rows, page_size, *strides, pos,
                                      slots, freqs, amp, layout, None)


@pytest.mark.parametrize("page_size", [16, 0])
def test_arguments(L, page_size):  # noqa: F811
    call = lambda **kw: append(L, **{**dict(page_size=page_size), **kw})
    for kw in (dict(dtype=2), dict(layout=2), dict(T=-1), dict(D=0), dict(rot=0), dict(amp=float("nan")), dict(Hk=0),
               dict(rows=-1), dict(slots=None), dict(pos=None), dict(freqs=None), dict(Q=None), dict(K=None),
               dict(V=None), dict(Qo=None), dict(Kc=None), dict(Vc=None)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(D=60), dict(D=264), dict(rot=24), dict(rot=80), dict(T=1 << 31), dict(Hq=70000)):
        assert call(**kw) == SHAPE, kw
    for kw in (dict(Q=ODD), dict(K=ODD), dict(V=ODD), dict(Qo=ODD), dict(Kc=ODD), dict(Vc=ODD), dict(pos=ODD),
               dict(slots=ODD), dict(freqs=ODD)):
        assert call(**kw) == ALIGN, kw
    assert call(T=0) == OK


def test_pages(L):  # noqa: F811
    assert append(L, page_size=-1) == INVALID
    assert append(L, page_size=1 << 31) == SHAPE
    for i in range(14):
        s = list(APPEND)
        s[i] += 2
        assert append(L, strides=s) == ALIGN, i
        s[i] = -8
        assert append(L, strides=s) == ALIGN, i
    for i in range(6, 14):  # an output's rows, heads or pages on one another
        s = list(APPEND)
        s[i] = 0
        assert append(L, strides=s) == INVALID, i
