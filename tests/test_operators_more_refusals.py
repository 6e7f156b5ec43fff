"""Refusals that come before any CUDA call: at the C entry points."""
from test_operators_abi import INVALID, L, OK, append, attention, rotary  # noqa: F401  (L is a fixture)


def test_heads_on_one_another_of_a_single_token(L):
    for f, n in ((rotary, 8), (append, 12)):
        for i in range(n // 2 + 1, n, 2):  # the outputs' head strides
            s = [256, 64] + [128, 64] * (n // 2 - 1)
            s[i] = 0
            assert f(L, T=1, strides=s) == INVALID, (f, i)


def test_scale_that_overflows_in_base_two(L):
    for scale in (2.5e38, 2.9e38, 3.4e38):
        assert attention(L, scale=scale) == INVALID, scale
    assert attention(L, scale=2.3e38, Tq=0) == OK
