"""Rotary angles at positions of any 64-bit size, within the bound that
include/w8a8.h states for them."""
from decimal import Decimal, getcontext

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("bits", [0, 20, 31, 40, 44, 48, 52, 56, 60, 62])
def test_angle_bound(w8a8, bits):
    """The angle is off by at most 2^-63 |p| turns (the turns per position are a sum
    of two numbers, each cut to a multiple of 2^-64), besides its own rounding to
    binary32; cos and sin move by no more than the angle does.  x = (1, 0) gives
    them directly: fp16 holds them with half a step of 2^-11."""
    getcontext().prec = 80
    two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")
    freqs = torch.tensor([1.0, 0.7390851332151607, 1e-3, 1e-5, 3.0, 0.1, 2.0 ** -20, 6.5], dtype=torch.float64,
                         device=DEV)
    base = 1 << bits
    pos = [base, -base, base + base // 3, -(base + base // 5) - 1]
    a = [[float((Decimal(p) * Decimal(f)) % two_pi) for f in freqs.tolist()] for p in pos]
    a = torch.tensor(a, dtype=torch.float64, device=DEV)
    x = torch.zeros(len(pos), 1, 16, dtype=torch.float16, device=DEV)
    x[..., :8] = 1
    got, _ = w8a8.rotary(x, None, torch.tensor(pos, device=DEV), freqs)
    want = torch.cat([a.cos(), a.sin()], -1)
    off = 6.3 * 2.0 ** -63 * torch.tensor([abs(p) for p in pos], dtype=torch.float64, device=DEV)[:, None]
    tol = off + 8e-7 + 2.0 ** -11 * want.abs() + 2.0 ** -25
    assert ((got[:, 0].double() - want).abs() <= tol).all()


@pytest.mark.parametrize("bits", [0, 31, 40, 44, 50])
def test_negative_frequencies_turn_back_as_far(w8a8, bits):
    """(-p)(-f) = p f to the bit, and p (-f) = -(p f) within the bounds of two
    calls (2^-32 of a turn each for the cut to 32 bits, then 8e-7 for binary32 and
    half a step of the type), also for frequencies so slow that 1 - f / 2 pi has no
    room for them."""
    torch.manual_seed(bits)
    x = torch.randn(6, 2, 16, device=DEV).to(torch.bfloat16)
    pos = (1 << bits) + torch.arange(6, device=DEV) * 977
    freqs = torch.tensor([1.0, 1e-2, 1e-3, 1e-5, 3e-7, 1e-9, 2.0 ** -20, 1e-12], dtype=torch.float64, device=DEV)
    ahead, _ = w8a8.rotary(x, None, pos, freqs)
    back, _ = w8a8.rotary(x, None, pos, freqs, inverse=True)
    assert torch.equal(w8a8.rotary(x, None, -pos, -freqs)[0], ahead)
    size = (x[..., :8].double().abs() + x[..., 8:].double().abs()).repeat(1, 1, 2)

    def tol(want):
        return 2 * (6.3 * 2.0 ** -32 + 8e-7) * size + 2 * 2.0 ** -8 * want.double().abs() * (1 + 2.0 ** -7)

    for got, want in ((w8a8.rotary(x, None, pos, -freqs)[0], back),
                      (w8a8.rotary(x, None, pos, -freqs, inverse=True)[0], ahead)):
        assert ((got.double() - want.double()).abs() <= tol(want)).all()
