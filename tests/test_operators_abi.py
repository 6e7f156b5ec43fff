"""Refusals of the attention, rotary and residual norm entry points: each
returns before any CUDA call, so this runs without a GPU."""
import ctypes

import pytest

P = ctypes.c_void_p
FAKE, ODD = P(0x1000), P(0x1002)  # never dereferenced
OK, INVALID, ALIGN, SHAPE = 0, 1, 2, 3


@pytest.fixture(scope="module")
def L():
    from w8a8_int8_linear_gb300 import build as b
    b.build()
    import w8a8_int8_linear_gb300 as w
    return w.lib()


def attention(L, Q=FAKE, K=FAKE, V=FAKE, O=FAKE, lse=None, cu_q=None, cu_k=None, k_lens=None, dtype=0, batch=1, Tq=4,
              Tk=4, Hq=4, Hk=2, D=64, strides=(256, 64, 128, 64, 128, 64, 256, 64), scale=0.125, causal=1, ws=FAKE,
              ws_bytes=1 << 30):
    return L.w8a8_attention(Q, K, V, O, lse, cu_q, cu_k, k_lens, dtype, batch, Tq, Tk, Hq, Hk, D, *strides, scale,
                            causal, ws, ws_bytes, None)


def test_attention(L):
    for kw in (dict(dtype=2), dict(dtype=-1), dict(batch=-1), dict(Tq=-1), dict(Tk=-1), dict(Hq=0), dict(Hk=0),
               dict(D=0), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(Q=None), dict(K=None), dict(V=None), dict(O=None)):
        assert attention(L, **kw) == INVALID, kw
    for kw in (dict(D=12), dict(D=136), dict(Hq=5), dict(batch=3), dict(batch=3, cu_q=FAKE), dict(batch=3, cu_k=FAKE),
               dict(Tq=1 << 31), dict(Tk=1 << 31)):
        assert attention(L, **kw) == SHAPE, kw
    for i in range(8):
        s = [256, 64, 128, 64, 128, 64, 256, 64]
        s[i] += 4
        assert attention(L, strides=s) == ALIGN
        s[i] = -8
        assert attention(L, strides=s) == ALIGN
    for kw in (dict(Q=ODD), dict(K=ODD), dict(V=ODD), dict(O=ODD), dict(lse=ODD), dict(cu_q=ODD), dict(cu_k=ODD),
               dict(k_lens=ODD)):
        assert attention(L, **kw) == ALIGN, kw
    assert attention(L, Tq=0, Q=None, O=None) == OK
    assert attention(L, batch=0) == OK


def rotary(L, Q=FAKE, K=FAKE, Qo=FAKE, Ko=FAKE, dtype=0, T=4, Hq=4, Hk=2, D=64, rot=32,
           strides=(256, 64, 128, 64, 256, 64, 128, 64), pos=FAKE, freqs=FAKE, amp=1.0, layout=0, inverse=0):
    return L.w8a8_rotary(Q, K, Qo, Ko, dtype, T, Hq, Hk, D, rot, *strides, pos, freqs, amp, layout, inverse, None)


def append(L, Q=FAKE, K=FAKE, V=FAKE, Qo=FAKE, Kc=FAKE, Vc=FAKE, dtype=0, T=4, Hq=4, Hk=2, D=64, rot=32, rows=10,
           strides=(256, 64) + (128, 64) * 2 + (256, 64) + (128, 64) * 2, pos=FAKE, slots=FAKE, freqs=FAKE, amp=1.0,
           layout=0):
    return L.w8a8_rotary_append(Q, K, V, Qo, Kc, Vc, dtype, T, Hq, Hk, D, rot, rows, *strides, pos, slots, freqs, amp,
                                layout, None)


def test_rotary(L):
    both = [dict(dtype=2), dict(layout=2), dict(T=-1), dict(D=0), dict(rot=0), dict(amp=float("nan")),
            dict(amp=float("inf")), dict(pos=None), dict(freqs=None), dict(Q=None), dict(K=None), dict(Qo=None)]
    for f, more in ((rotary, [dict(Hq=-1), dict(Hk=-1), dict(Ko=None)]),
                    (append, [dict(Hk=0), dict(rows=-1), dict(slots=None), dict(V=None), dict(Kc=None),
                              dict(Vc=None)])):
        for kw in both + more:
            assert f(L, **kw) == INVALID, kw
        for kw in (dict(D=60), dict(D=264), dict(rot=24), dict(rot=80), dict(T=1 << 31), dict(Hq=70000)):
            assert f(L, **kw) == SHAPE, kw
        for kw in (dict(Q=ODD), dict(K=ODD), dict(Qo=ODD), dict(pos=ODD), dict(freqs=ODD)):
            assert f(L, **kw) == ALIGN, kw
        n = 8 if f is rotary else 12
        for i in range(n):
            s = [256, 64] + [128, 64] * (n // 2 - 1)
            s[i] += 2
            assert f(L, strides=s) == ALIGN
        assert f(L, T=0) == OK
    assert rotary(L, Hq=0, Hk=0) == OK
    assert append(L, slots=ODD) == ALIGN


def norm(L, X=FAKE, B=FAKE, H=FAKE, dtype=0, bg=None, g=None, be=None, gate=None, sc=None, sh=None, stride=0, rpg=0,
         alpha=1.0, eps=1e-6, kind=0, M=4, K=64, Y=FAKE, Xq=FAKE, Ximg=FAKE, sx=FAKE):
    return L.w8a8_residual_norm_quant(X, B, H, dtype, bg, g, be, gate, sc, sh, stride, rpg, alpha, eps, kind, M, K, Y,
                                      Xq, Ximg, sx, None)


def test_residual_norm(L):
    for kw in (dict(dtype=1), dict(kind=2), dict(M=-1), dict(K=0), dict(rpg=-1), dict(stride=-8), dict(eps=-1.0),
               dict(eps=float("nan")), dict(alpha=float("nan")), dict(X=None), dict(B=None), dict(H=None),
               dict(sx=None), dict(Xq=None, Ximg=None)):
        assert norm(L, **kw) == INVALID, kw
    for kw in (dict(K=12), dict(K=16392), dict(M=1 << 31)):
        assert norm(L, **kw) == SHAPE, kw
    for name in ("X", "B", "H", "bg", "g", "be", "gate", "sc", "sh", "Y", "Xq", "Ximg", "sx"):
        assert norm(L, **{name: ODD}) == ALIGN, name
    assert norm(L, stride=4) == ALIGN
    assert norm(L, M=0, X=None) == OK


def test_workspace_sizes_need_a_device(L):
    import torch
    if torch.cuda.is_available():
        size, zeroed = L.w8a8_attention_workspace_size(), L.w8a8_attention_workspace_zeroed()
        assert size > zeroed > 0 and size % 256 == 0 and zeroed % 256 == 0
    else:
        assert L.w8a8_attention_workspace_size() == 0 and L.w8a8_attention_workspace_zeroed() == 0


def test_rotary_outputs_on_one_another(L):
    for f, n in ((rotary, 8), (append, 12)):
        for i in range(n // 2, n):
            s = [256, 64] + [128, 64] * (n // 2 - 1)
            s[i] = 0
            assert f(L, strides=s) == INVALID, (f, i)
