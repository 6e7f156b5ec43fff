"""Refusals that come before any CUDA call: at the C entry points."""
from test_operators_abi import INVALID, L, append, rotary  # noqa: F401  (L is a fixture)


def test_heads_on_one_another_of_a_single_token(L):
    for f, n in ((rotary, 8), (append, 12)):
        for i in range(n // 2 + 1, n, 2):  # the outputs' head strides
            s = [256, 64] + [128, 64] * (n // 2 - 1)
            s[i] = 0
            assert f(L, T=1, strides=s) == INVALID, (f, i)
