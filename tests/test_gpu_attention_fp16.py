"""fp16 weights over their whole range: far below the row's largest, where fp16
itself has no normal numbers, and at the largest that the kernels hold."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
FP16 = torch.float16


@pytest.mark.parametrize("place", ["first", "last", "middle"])
@pytest.mark.parametrize("n,m,group,d", [(1, 131072, 4, 128), (6, 65536, 4, 64), (12, 65536, 4, 128), (3600, 16384, 1, 128),
                                         (3600, 16384, 1, 64)])
def test_fp16_weights_far_below_the_largest(w8a8, n, m, group, d, place):
    """One key of weight 1 and value 0, all others of weight 2^-26 (less than
    half of fp16's smallest number) and values near 1: the output is what these
    add up to, n 2^-26.

    Tolerance, as for attention elsewhere (half a step u = 2^-11 for the weights
    and the output, 2 dt for the scores, 2^-20 and m 2^-24 for the exponentials
    and the sums in binary32), but what fp16 leaves of a weight below its normal
    range: the kernels hold the largest weight of a row at 2^7 at least, so half
    of the smallest number, 2^-25, is 2^-32 of it."""
    g = torch.Generator(device=DEV).manual_seed(m + d)
    q = torch.zeros(n, group, d, dtype=FP16, device=DEV)
    q[..., 0] = 8.0
    at = {"first": 3, "last": m - 5, "middle": m // 2 + 77}[place]
    k = torch.zeros(m, 1, d, dtype=FP16, device=DEV)
    k[..., 0] = -9.0
    k[at, 0, 0] = 9.0
    v = (1 + 0.1 * torch.randn(m, 1, d, generator=g, device=DEV)).to(FP16)
    v[at] = 0
    o, lse = w8a8.attention(q, k, v, causal=False, scale=0.125, lse=True)
    t = torch.full((m,), -9.0, dtype=torch.float64, device=DEV)
    t[at] = 9.0
    w = torch.softmax(t, 0)
    want = w @ v[:, 0].double()
    dt = (d + 4) * 2.0 ** -24 * 9.0
    tol = (2.0 ** -11 + 2 * dt + 2.0 ** -20 + m * 2.0 ** -24) * want + 2.0 ** -11 * want \
        + 2.0 ** -32 * v[:, 0].double().sum(0)
    assert (want > 10 * tol).all()  # otherwise zeros would pass
    assert ((o.double() - want).abs() <= tol).all(), float(((o.double() - want).abs() - tol).max())
    want_lse = float(torch.logsumexp(t, 0))
    assert ((lse.double() - want_lse).abs() <= 2 * dt + 2.0 ** -20 + m * 2.0 ** -24 + abs(want_lse) * 2.0 ** -22).all()
    assert w8a8.get_device_error() == (0, 0)


@pytest.mark.parametrize("n,m", [(2, 5000), (1100, 1500)])
def test_fp16_weights_at_their_largest(w8a8, n, m):
    """The largest values of fp16 under the largest weights that the kernels hold:
    scores that rise by 5.5 (2^7.9 in weight) after the first tile of 128 keys.  All V are 60000, so that every output is, up to the weights'
    rounding (half a step each, 2^-11, in the same direction at worst), the sums'
    (m 2^-24) and its own (16 for a number below 65536)."""
    q = torch.zeros(n, 4, 64, dtype=FP16, device=DEV)
    q[..., 0] = 1.0
    k = torch.zeros(m, 1, 64, dtype=FP16, device=DEV)
    k[128:, 0, 0] = 5.5
    v = torch.full((m, 1, 64), 60000.0, dtype=FP16, device=DEV)
    o = w8a8.attention(q, k, v, causal=False, scale=1.0)
    assert ((o.double() - 60000).abs() <= 60000 * (2.0 ** -11 + m * 2.0 ** -24 + 2.0 ** -20) + 16).all()


@pytest.mark.parametrize("queries", [1, 5, 12])
def test_fp16_weights_below_the_normal_range_over_caches(w8a8, queries):
    """240 caches of 8192 keys, each with eight keys of weight 1 and value 0 (so
    that every warp which begins a sequence meets one); the others weigh about
    1.5 2^-24, which fp16 would hold as 1 or 2 times 2^-24.  Tolerance as above."""
    batch, m, d = 240, 8192, 64
    q = torch.zeros(batch * queries, 4, d, dtype=FP16, device=DEV)
    q[..., 0] = 8.0
    k = torch.zeros(m, d, dtype=FP16, device=DEV)
    k[:, 0] = -8.234375
    k[0:128:16, 0] = 8.0
    v = (1 + 0.1 * torch.randn(m, d, generator=torch.Generator(device=DEV).manual_seed(2), device=DEV)).to(FP16)
    v[0:128:16] = 0
    kc, vc = (x[None].expand(batch, m, d).reshape(batch * m, 1, d) for x in (k, v))
    o, lse = w8a8.attention(q, kc, vc, batch=batch, causal=False, scale=0.125, lse=True)
    t = k[:, 0].double()
    want = torch.softmax(t, 0) @ v.double()
    dt = (d + 4) * 2.0 ** -24 * 8.25
    tol = (2.0 ** -11 + 2 * dt + 2.0 ** -20 + m * 2.0 ** -24) * want + 2.0 ** -11 * want \
        + 2.0 ** -32 * v.double().sum(0) / 8 + 2.0 ** -25
    assert (want > 100 * tol).all()
    assert ((o.double() - want).abs() <= tol).all(), float(((o.double() - want).abs() / want).max())
    want_lse = float(torch.logsumexp(t, 0))
    assert ((lse.double() - want_lse).abs() <= 2 * dt + 2.0 ** -20 + m * 2.0 ** -24 + abs(want_lse) * 2.0 ** -22).all()
    assert w8a8.get_device_error() == (0, 0)
