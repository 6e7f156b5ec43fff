"""Norms of the query and key heads with rotary positions, against the formula in
64 bits.

Tolerance.  The sum of squares of D terms in binary32 is off by at most
(D + 1) 2^-24 relative in any order, its root by half of that; the mean, eps, the
reciprocal root (2 units) and the two products add 8 roundings: y is off by
(D / 2 + 8) 2^-24 |y|.  LayerNorm's mean is off by D 2^-24 mean|x|, that is in y
twice of it (in the difference, and through the variance) over the deviation.
Turning adds 8e-7 (|y1| + |y2|) as test_gpu_rotary derives, then one rounding to
the type."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, FP16 = torch.bfloat16, torch.float16


def exact(x, gamma, kind, w8a8, eps, positions, freqs, layout, amp):
    """x [T, H, D] normed and turned in 64 bits, and its tolerance."""
    d, rot = x.shape[-1], 2 * freqs.numel()
    y = x.double()
    mean_abs = y.abs().mean(-1, keepdim=True)
    if kind == w8a8.LAYER_NORM:
        y = y - y.mean(-1, keepdim=True)
    r = 1 / (y.square().mean(-1, keepdim=True) + eps).sqrt()
    g = 1.0 if gamma is None else gamma.double()
    y = y * r * g
    off = (d / 2 + 8) * 2.0 ** -24 * y.abs()
    if kind == w8a8.LAYER_NORM:
        shift = d * 2.0 ** -24 * mean_abs * r
        off = off + shift * (torch.ones_like(y) * g).abs() + shift * y.abs()
    a, b = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    angle = positions.double()[:, None] * freqs[None]
    c, s = (amp * angle.cos())[:, None], (amp * angle.sin())[:, None]
    out, tol = y.clone(), off.clone()
    p, q = y[..., a], y[..., b]
    out[..., a], out[..., b] = p * c - q * s, q * c + p * s
    tol[..., a] = tol[..., b] = amp * (off[..., a] + off[..., b] + 8e-7 * (p.abs() + q.abs()))
    fi = torch.finfo(x.dtype)
    return out, tol * (1 + fi.eps) + fi.eps / 2 * out.abs() + fi.tiny * fi.eps


def close(got, *args):
    y, tol = exact(*args)
    bad = (got.double() - y).abs() > tol
    assert not bad.any(), (bad.nonzero()[:3].tolist(), float(((got.double() - y).abs() - tol).max()))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("kind", ["RMS_NORM", "LAYER_NORM"])
@pytest.mark.parametrize("t,hq,hk,d,rot,dtype,page", [
    (1, 1, 1, 16, 16, BF16, 8), (3, 40, 8, 128, 128, BF16, 16), (65, 5, 5, 64, 32, FP16, 64), (7, 32, 1, 256, 256, BF16, 1),
    (129, 3, 2, 80, 32, FP16, 24), (33, 8, 2, 192, 64, BF16, 0), (2, 12, 4, 96, 96, FP16, 16), (301, 7, 0, 128, 64, BF16, 0),
    (11, 3, 3, 72, 16, BF16, 5), (9, 2, 1, 24, 16, FP16, 3), (5, 70, 70, 40, 32, BF16, 7), (2500, 6, 2, 128, 128, BF16, 64)])
def test_norm_rotary(w8a8, t, hq, hk, d, rot, dtype, page, kind, layout):
    g = torch.Generator(device=DEV).manual_seed(t + d)
    kind = getattr(w8a8, kind)
    qkv = (torch.randn(t, hq + 2 * hk, d, generator=g, device=DEV) * 3 + 0.5).to(dtype)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    k = k if hk else None
    qg = torch.randn(d, generator=g, device=DEV).to(dtype)
    # every key head its own row, part of something wider
    kg = torch.randn(hk, d + 8, generator=g, device=DEV).to(dtype)[:, :d] if hk else None
    pos = torch.randint(-1000, 1 << 20, (t,), generator=g, device=DEV)
    freqs = w8a8.rotary_frequencies(rot)
    more = (kind, w8a8, 1e-5, pos, freqs, layout, 1.25)
    opts = dict(q_gamma=qg, k_gamma=kg, eps=1e-5, kind=kind, layout=layout, amplitude=1.25)
    keep = qkv.clone()
    q1, k1 = w8a8.qk_norm_rotary(q, k, pos, freqs, **opts)
    assert torch.equal(qkv, keep)
    close(q1, q, qg, *more)
    if hk:
        close(k1, k, kg, *more)
        # K and V of every other token into cache rows, from the back
        rows = 2 * t + 3
        if page:
            rows = -(-rows // page) * page
            wide = torch.full((rows // page, 2, page, hk, d), 9.0, dtype=dtype, device=DEV)
            kc, vc = wide[:, 0], wide[:, 1]
        else:
            kc = torch.full((rows, hk, d), 9.0, dtype=dtype, device=DEV)
            vc = torch.full_like(kc, 9.0)
        slots = torch.arange(2 * t, 0, -2, device=DEV)
        slots[::2] = torch.where(torch.arange(len(slots[::2]), device=DEV) % 2 == 0, -1, rows)
        q2 = w8a8.qk_norm_rotary_append(q, k, v, pos, freqs, kc, vc, slots, **opts)
        assert torch.equal(q2, q1)
        want_k = torch.full((rows, hk, d), 9.0, dtype=dtype, device=DEV)
        want_v = want_k.clone()
        want_k[slots[1::2]], want_v[slots[1::2]] = k1[1::2], v[1::2]
        assert torch.equal(kc.reshape(rows, hk, d), want_k) and torch.equal(vc.reshape(rows, hk, d), want_v)
    # in place on the views
    w8a8.qk_norm_rotary(q, k, pos, freqs, q_out=q, k_out=k, **opts)
    assert torch.equal(q, q1) and (k is None or torch.equal(k, k1))
    assert torch.equal(qkv[:, hq + hk:], keep[:, hq + hk:])


def test_without_gamma_and_of_other_sizes(w8a8):
    """No gamma; tiny, huge, zero and constant heads."""
    freqs = w8a8.rotary_frequencies(64)
    pos = torch.arange(6, device=DEV)
    x = torch.randn(6, 3, 64, device=DEV)
    x[0] *= 1e-6
    x[1] *= 1e15
    x[2] = 0
    x[3] = 5.0
    x = x.to(BF16)
    for kind in (w8a8.RMS_NORM, w8a8.LAYER_NORM):
        y, k = w8a8.qk_norm_rotary(x, None, pos, freqs, kind=kind)
        assert k is None
        close(y, x, None, kind, w8a8, 1e-6, pos, freqs, "half", 1.0)
        assert (y[2] == 0).all()
    y, _ = w8a8.qk_norm_rotary(x, None, pos, freqs, eps=0.0)
    assert torch.isfinite(y[[0, 1, 3, 4, 5]]).all()


def test_a_head_that_is_not_finite_stays_alone(w8a8):
    freqs = w8a8.rotary_frequencies(128)
    pos = torch.arange(4, device=DEV)
    x = torch.randn(4, 9, 128, device=DEV).to(BF16)
    base, _ = w8a8.qk_norm_rotary(x, x, pos, freqs)
    for value in (math.nan, math.inf):
        y = x.clone()
        y[2, 5, 77] = value
        got, _ = w8a8.qk_norm_rotary(y, y, pos, freqs)
        assert not torch.isfinite(got[2, 5, 77])
        got[2, 5] = base[2, 5]
        assert torch.equal(got, base)


def test_captured(w8a8):
    freqs = w8a8.rotary_frequencies(64)
    q, k, v = (torch.randn(5, h, 64, device=DEV).to(BF16) for h in (4, 2, 2))
    pos, slots = torch.arange(5, device=DEV), torch.tensor([9, 3, -1, 31, 0], device=DEV)
    caches = [torch.zeros(2, 16, 2, 64, dtype=BF16, device=DEV) for _ in range(4)]
    w8a8.qk_norm_rotary_append(q, k, v, pos, freqs, caches[2], caches[3], slots)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = w8a8.qk_norm_rotary_append(q, k, v, pos, freqs, caches[0], caches[1], slots)
    for step in range(3):
        q.normal_()
        k.normal_()
        pos += 1000
        slots.copy_((slots + 1).clamp(max=31))
        graph.replay()
        assert torch.equal(out, w8a8.qk_norm_rotary_append(q, k, v, pos, freqs, caches[2], caches[3], slots))
        for a, b in zip(caches[:2], caches[2:]):
            i = slots[slots >= 0]
            assert torch.equal(a.flatten(0, 1)[i[:2]], b.flatten(0, 1)[i[:2]])


def test_rows_past_32_bits(w8a8):
    page, hk, d = 32, 4, 128
    pages = (5 << 30) // (page * hk * d * 2) + 1
    kc, vc = (torch.zeros(pages, page, hk, d, dtype=BF16, device=DEV) for _ in range(2))
    q, k, v = (torch.randn(3, h, d, device=DEV).to(BF16) for h in (8, hk, hk))
    pos = torch.arange(3, device=DEV)
    slots = torch.tensor([pages * page - 1, 5, pages * page // 2 + 3], device=DEV)
    freqs = w8a8.rotary_frequencies(d)
    w8a8.qk_norm_rotary_append(q, k, v, pos, freqs, kc, vc, slots)
    _, k1 = w8a8.qk_norm_rotary(q, k, pos, freqs)
    assert torch.equal(kc.flatten(0, 1)[slots], k1) and torch.equal(vc.flatten(0, 1)[slots], v)


def test_nothing_to_do(w8a8):
    freqs = w8a8.rotary_frequencies(64)
    z = torch.empty(0, dtype=torch.int64, device=DEV)
    x = torch.empty(0, 4, 64, dtype=BF16, device=DEV)
    q, k = w8a8.qk_norm_rotary(x, x, z, freqs)
    assert q.shape == k.shape == (0, 4, 64)
    cache = torch.zeros(2, 8, 4, 64, dtype=BF16, device=DEV)
    assert w8a8.qk_norm_rotary_append(x, x, x, z, freqs, cache, cache.clone(), z).shape == (0, 4, 64)
    # no query heads: only K and V
    one = torch.zeros(1, dtype=torch.int64, device=DEV)
    none, kv = torch.empty(1, 0, 64, dtype=BF16, device=DEV), torch.randn(1, 4, 64, device=DEV).to(BF16)
    kc, vc = cache.clone(), cache.clone()
    assert w8a8.qk_norm_rotary_append(none, kv, kv, one + 1, freqs, kc, vc, one + 9).shape == (1, 0, 64)
    assert torch.equal(vc[1, 1], kv[0]) and torch.equal(kc[1, 1], w8a8.qk_norm_rotary(kv, None, one + 1, freqs)[0][0])
    # a cache of no rows is refused, as by rotary_append
    empty = cache[:0]
    with pytest.raises(w8a8.W8A8Error):
        w8a8.qk_norm_rotary_append(kv, kv, kv, one, freqs, empty, empty.clone(), one)


def test_values_of_v_are_copied_bit_for_bit(w8a8):
    freqs = w8a8.rotary_frequencies(64)
    bits = torch.randint(-32768, 32768, (40, 2, 64), dtype=torch.int16, device=DEV)
    v = bits.view(BF16)
    kc, vc = (torch.zeros(3, 16, 2, 64, dtype=BF16, device=DEV) for _ in range(2))
    k = torch.randn(40, 2, 64, device=DEV).to(BF16)
    slots = torch.randperm(48, device=DEV)[:40]
    w8a8.qk_norm_rotary_append(k, k, v, slots, freqs, kc, vc, slots)
    assert torch.equal(vc.flatten(0, 1)[slots].view(torch.int16), bits)
