"""The "yarn" table's two ramps, against the formulas pair by pair."""
import math

import pytest
import torch

from w8a8_int8_linear_gb300 import rotary_frequencies

CASES = [(128, 10000.0, 8.0, 16384, 32.0, 1.0), (64, 500.0, 4.0, 2048, 32.0, 1.0), (96, 1e6, 40.0, 4096, 32.0, 1.0),
         (32, 150000.0, 32.0, 4096, 20.0, 2.0), (16, 10000.0, 2.0, 100, 64.0, 8.0)]


def table(ramp, r, base, factor, length, fast, slow, **kw):
    return rotary_frequencies(r, base, "yarn", factor, original_length=length, fast=fast, slow=slow, device="cpu",
                              **ramp, **kw).tolist()


@pytest.mark.parametrize("r,base,factor,length,fast,slow", CASES)
def test_ramp_over_turns(r, base, factor, length, fast, slow):
    for ramp in ({}, dict(ramp="turns")):
        for k, got in enumerate(table(ramp, r, base, factor, length, fast, slow)):
            f = base ** (-2 * k / r)
            keep = min(1.0, max(0.0, (length * f / (2 * math.pi) - slow) / (fast - slow)))
            assert got == pytest.approx(f * keep + f / factor * (1 - keep), rel=1e-12)


@pytest.mark.parametrize("r,base,factor,length,fast,slow", CASES)
def test_ramp_over_pairs(r, base, factor, length, fast, slow):
    """Linear in the pair's index from the last pair with `fast` turns, rounded
    down, to the first with `slow`, rounded up."""
    def pair(turns):  # the (fractional) pair that turns so often in `length` positions
        return r * math.log(length / (2 * math.pi * turns)) / (2 * math.log(base))

    low, high = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), r - 1)
    for k, got in enumerate(table(dict(ramp="pairs"), r, base, factor, length, fast, slow)):
        f = base ** (-2 * k / r)
        stretched = min(1.0, max(0.0, (k - low) / max(high - low, 1e-3)))
        assert got == pytest.approx(f / factor * stretched + f * (1 - stretched), rel=1e-12)


def test_the_ramps_differ_and_share_their_ends():
    turns, pairs = (torch.tensor(table(dict(ramp=x), *CASES[0])) for x in ("turns", "pairs"))
    plain = 10000.0 ** -(torch.arange(0, 128, 2, dtype=torch.float64) / 128)
    for t in (turns, pairs):
        assert t[0] == plain[0] and t[-1] == pytest.approx(float(plain[-1] / 8))
    assert (turns / pairs - 1).abs().max() > 0.3


def test_refusals():
    with pytest.raises(ValueError, match="ramp must be 'turns' or 'pairs'"):
        table(dict(ramp="other"), *CASES[0])
    for ramp in ("turns", "pairs"):
        with pytest.raises(ValueError):
            rotary_frequencies(16, scaling="yarn", factor=2.0, ramp=ramp, device="cpu")
        with pytest.raises(ValueError):
            rotary_frequencies(16, scaling="yarn", factor=2.0, original_length=100, fast=1.0, slow=1.0, ramp=ramp,
                               device="cpu")
    with pytest.raises(ValueError):
        rotary_frequencies(16, scaling="yarn", factor=2.0, original_length=100, slow=0.0, ramp="pairs", device="cpu")
    assert rotary_frequencies(16, scaling="yarn", factor=2.0, original_length=100, slow=0.0, device="cpu").shape == (8,)
