"""Rotary positions against the formula in 64 bits.

Tolerance: the angle in half turns is rounded to binary32 once (2^-24
relative, at most pi: 2e-7 radians), cos and sin are within 2 units of 2^-24,
and the products and sum of the pair add 2^-23 (|x| + |y|); with the
amplitude a that is 8e-7 a (|x| + |y|), then one rounding to the type."""
import math
from decimal import Decimal, getcontext

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, FP16 = torch.bfloat16, torch.float16


def exact(x, cos, sin, rot, layout):
    """x [T, H, D] turned in 64 bits, and the tolerance without the amplitude's share."""
    y = x.double().clone()
    a, b = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    p, q = x.double()[..., a], x.double()[..., b]
    y[..., a] = p * cos[:, None] - q * sin[:, None]
    y[..., b] = q * cos[:, None] + p * sin[:, None]
    size = torch.zeros_like(y)
    size[..., a] = size[..., b] = p.abs() + q.abs()
    return y, size


def check(got, x, cos, sin, rot, layout, amp):
    y, size = exact(x, cos * amp, sin * amp, rot, layout)
    fi = torch.finfo(x.dtype)
    tol = 8e-7 * amp * size * (1 + fi.eps) + fi.eps / 2 * y.abs() + fi.tiny * fi.eps
    assert ((got.double() - y).abs() <= tol).all()
    assert torch.equal(got[..., rot:], x[..., rot:])


def angles(positions, freqs):
    a = positions.double()[:, None] * freqs[None]
    return a.cos(), a.sin()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("t,hq,hk,d,rot,dtype", [
    (1, 1, 1, 16, 16, BF16), (3, 40, 8, 128, 128, BF16), (65, 5, 5, 64, 32, FP16), (7, 32, 1, 256, 256, BF16),
    (129, 3, 2, 80, 32, FP16), (33, 8, 2, 192, 64, BF16), (2, 12, 4, 96, 96, FP16), (301, 7, 0, 128, 64, BF16)])
def test_rotary(w8a8, t, hq, hk, d, rot, layout, dtype):
    g = torch.Generator(device=DEV).manual_seed(t + d)
    qkv = torch.randn(t, hq + 2 * hk, d, generator=g, device=DEV).to(dtype)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    k = k if hk else None
    pos = torch.randint(-1000, 1 << 20, (t,), generator=g, device=DEV)
    freqs = w8a8.rotary_frequencies(rot)
    cos, sin = angles(pos, freqs)
    keep = qkv.clone()
    q1, k1 = w8a8.rotary(q, k, pos, freqs, layout=layout, amplitude=1.25)
    assert torch.equal(qkv, keep)
    check(q1, q, cos, sin, rot, layout, 1.25)
    if hk:
        check(k1, k, cos, sin, rot, layout, 1.25)
        # K and V of every other token into cache rows, from the back
        kc = torch.full((2 * t + 3, hk, d), 9.0, dtype=dtype, device=DEV)
        vc = torch.full_like(kc, 9.0)
        slots = torch.arange(2 * t, 0, -2, device=DEV)
        slots[::2] = torch.where(torch.arange(len(slots[::2]), device=DEV) % 2 == 0, -1, 2 * t + 3)
        q2 = w8a8.rotary_append(q, k, v, pos, freqs, kc, vc, slots, layout=layout, amplitude=1.25)
        assert torch.equal(q2, q1)
        want_k, want_v = torch.full_like(kc, 9.0), torch.full_like(vc, 9.0)
        want_k[slots[1::2]], want_v[slots[1::2]] = k1[1::2], v[1::2]
        assert torch.equal(kc, want_k) and torch.equal(vc, want_v)
    # in place on the views, and back
    w8a8.rotary(q, k, pos, freqs, layout=layout, amplitude=1.25, q_out=q, k_out=k)
    assert torch.equal(q, q1) and (k is None or torch.equal(k, k1))
    assert torch.equal(qkv[:, hq + hk:], keep[:, hq + hk:])
    q3, _ = w8a8.rotary(keep[:, :hq], None, pos, freqs, layout=layout, inverse=True)
    check(q3, keep[:, :hq], cos, -sin, rot, layout, 1.0)


def test_far_positions(w8a8):
    """Positions at which the product p f no longer fits a double: against the
    angle reduced in 60 decimal digits."""
    getcontext().prec = 60
    two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494")
    freqs = torch.tensor([1.0, 0.7390851332151607, 1e-3, 1e-5, 3.0, 0.1, 2.0 ** -20, 6.5], dtype=torch.float64,
                         device=DEV)
    pos = [0, 1, -1, 12345678, (1 << 31) + 7, (1 << 40) - 1, -(1 << 36) + 5]
    a = [[float((Decimal(p) * Decimal(f)) % two_pi) for f in freqs.tolist()] for p in pos]
    a = torch.tensor(a, dtype=torch.float64, device=DEV)
    x = torch.randn(len(pos), 3, 16, device=DEV).to(BF16)
    got, _ = w8a8.rotary(x, None, torch.tensor(pos, device=DEV), freqs)
    check(got, x, a.cos(), a.sin(), 16, "half", 1.0)


def test_gradient_is_the_inverse(w8a8):
    """The gradient of sum(g * rotary(x)) is rotary^-1(g): against the formula
    (transpose of the turn) and against differences of the 64-bit forward."""
    torch.manual_seed(5)
    pos = torch.arange(5, device=DEV) * 1000
    freqs = w8a8.rotary_frequencies(32)
    cos, sin = angles(pos, freqs)
    x, g = (torch.randn(5, 2, 32, device=DEV).to(FP16) for _ in range(2))
    back, _ = w8a8.rotary(g, None, pos, freqs, inverse=True)
    check(back, g, cos, -sin, 32, "half", 1.0)
    h = 1e-3
    for i in (0, 7, 19, 31):
        up, down = x.double().clone(), x.double().clone()
        up[..., i] += h
        down[..., i] -= h
        diff = (g.double() * (exact(up, cos, sin, 32, "half")[0] - exact(down, cos, sin, 32, "half")[0])).sum(-1) / (2 * h)
        size = g.double().abs().sum(-1)
        assert ((back[..., i].double() - diff).abs() <= 2.0 ** -11 * diff.abs() + 1e-6 * size + 1e-6).all()


def test_frequencies(w8a8):
    f = w8a8.rotary_frequencies(64, base=500.0)
    assert f.dtype == torch.float64 and f.shape == (32,)
    assert torch.allclose(f, torch.tensor([500.0 ** (-2 * k / 64) for k in range(32)], dtype=torch.float64,
                                          device=DEV), rtol=1e-14, atol=0)
    assert torch.equal(w8a8.rotary_frequencies(64, 500.0, "linear", 4.0), f / 4)
    n = w8a8.rotary_frequencies(64, 500.0, "ntk", 4.0)
    assert n[0] == 1 and abs(float(n[-1] / f[-1]) - 0.25) < 1e-12
    y = w8a8.rotary_frequencies(64, 500.0, "yarn", 4.0, original_length=2048)
    turns = 2048 * f / (2 * math.pi)
    assert torch.equal(y[turns >= 32], f[turns >= 32]) and torch.allclose(y[turns <= 1], f[turns <= 1] / 4)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and (y[mid] < f[mid]).all() and (y[mid] > f[mid] / 4).all()
    for kw in (dict(rot_dim=3), dict(rot_dim=0), dict(rot_dim=8, scaling="other"), dict(rot_dim=8, factor=0.5),
               dict(rot_dim=8, scaling="yarn", factor=2.0), dict(rot_dim=2, scaling="ntk", factor=2.0)):
        with pytest.raises(ValueError):
            w8a8.rotary_frequencies(**kw)


def test_refusals(w8a8):
    q = torch.zeros(4, 2, 32, dtype=BF16, device=DEV)
    pos = torch.arange(4, device=DEV)
    f = w8a8.rotary_frequencies(32)
    cases = [
        (TypeError, lambda: w8a8.rotary(q.float(), None, pos, f)),
        (TypeError, lambda: w8a8.rotary(q, q.half(), pos, f)),
        (TypeError, lambda: w8a8.rotary(q, None, pos.int(), f)),
        (TypeError, lambda: w8a8.rotary(q, None, pos, f.float())),
        (ValueError, lambda: w8a8.rotary(q, None, pos[:3], f)),
        (ValueError, lambda: w8a8.rotary(q, None, pos, f, layout="other")),
        (ValueError, lambda: w8a8.rotary(q, None, pos, f, q_out=q[:2])),
        (ValueError, lambda: w8a8.rotary(q, q[:2], pos, f)),
        (ValueError, lambda: w8a8.rotary_append(q, q, q[:, :1], pos, f, q, q, pos)),
        (w8a8.W8A8Error, lambda: w8a8.rotary(q, None, pos, w8a8.rotary_frequencies(48))),
        (w8a8.W8A8Error, lambda: w8a8.rotary(q, None, pos, w8a8.rotary_frequencies(24))),
        (w8a8.W8A8Error, lambda: w8a8.rotary(q, None, pos, f, amplitude=math.nan)),
    ]
    for err, call in cases:
        with pytest.raises(err):
            call()
    assert w8a8.rotary(q[:0], None, pos[:0], f)[0].shape == (0, 2, 32)
