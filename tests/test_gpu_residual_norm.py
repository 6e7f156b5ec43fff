"""residual_norm_quant against its formula in 64 bits.

Tolerance (u = 2^-24): the sums run over at most 80 rounded additions per
element (8 per chunk and at most 8 chunks of a thread, then two trees of 5),
so a mean square is off by 90 u relative, the reciprocal root by 50 u, the
mean by 90 u mean|h|; each further product or sum adds u of its size.
  h: 60 u on the normed branch, 4 u on each term;
  y: 60 u of the terms' sizes plus the error that h brings, r |g| dh;
then half a step of the output's type.  A code is off by at most half a step
plus what y and the scale are off by."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16
U = 2.0 ** -24


def exact(x, b, gamma, beta, eps, layer, alpha, gate, branch_gamma, scale, shift, rows_per_group):
    """h, y in 64 bits and the absolute error bounds of their binary32 values."""
    m, k = x.shape
    eps = float(torch.tensor(eps, dtype=torch.float32))
    row = torch.arange(m, device=DEV) // rows_per_group if rows_per_group else torch.zeros(m, dtype=torch.long, device=DEV)

    def per_row(t):
        return t.double().reshape(-1, k)[row]

    br, db = b.double(), 0.0
    if branch_gamma is not None:
        br = br / (br.square().mean(1, keepdim=True) + eps).sqrt() * branch_gamma.double()
        db = 60 * U * br.abs()
    if gate is not None:
        br = br * per_row(gate)
        db = db * per_row(gate).abs() if branch_gamma is not None else 0.0
    ax = float(torch.tensor(alpha, dtype=torch.float32)) * x.double()
    h = ax + br
    dh = db + 4 * U * (ax.abs() + br.abs())
    mu = h.mean(1, keepdim=True) if layer else 0.0
    dmu = 90 * U * h.abs().mean(1, keepdim=True) + dh.mean(1, keepdim=True) if layer else 0.0
    r = 1 / ((h - mu).square().mean(1, keepdim=True) + eps).sqrt()
    dr = 50 * U + (dh * (h - mu).abs()).mean(1, keepdim=True) * r * r * 2  # relative
    g = gamma.double() if gamma is not None else torch.ones(k, dtype=torch.float64, device=DEV)
    n = (h - mu) * r * g
    dn = r * g.abs() * (dh + dmu) + n.abs() * (dr + 8 * U)
    if beta is not None:
        n = n + beta.double()
        dn = dn + 2 * U * n.abs()
    if scale is not None:
        dn = dn * (1 + per_row(scale)).abs() + 4 * U * (n.abs() + (n * per_row(scale)).abs())
        n = n * (1 + per_row(scale))
    if shift is not None:
        n = n + per_row(shift)
        dn = dn + 2 * U * (n.abs() + per_row(shift).abs())
    return h, dh, n, dn


def half_step(t):
    return torch.finfo(t).eps / 2


CASES = [
    # rows, width, kind, x dtype, branch norm, gamma, beta, modulation groups (None: none), alpha
    (1, 8, "rms", BF16, False, False, False, None, 1.0), (3, 64, "layer", BF16, True, True, True, 1, 0.5),
    (5, 2040, "rms", torch.float32, True, True, False, None, 1.0), (7, 2056, "layer", BF16, False, False, False, 2, 1.0),
    (33, 5120, "rms", BF16, False, True, False, None, 1.0), (4, 5120, "rms", BF16, True, True, False, None, 0.5),
    (10, 4096, "layer", torch.float32, False, False, False, 3, 1.0), (9, 8192, "layer", torch.float32, True, True, True, 4, -1.5),
    (6, 8200, "rms", BF16, False, True, True, 2, 1.0), (2, 16384, "layer", BF16, True, True, False, None, 1.0),
    (257, 1000, "rms", BF16, True, True, False, 5, 0.25), (2500, 1000, "layer", BF16, True, True, True, 7, 1.0),
    (1300, 5120, "rms", BF16, True, True, False, None, 1.0), (1111, 8192, "layer", torch.float32, False, True, True, 2, 0.5),
    (700, 16384, "rms", torch.float32, True, True, False, 2, 1.0), (3001, 64, "rms", BF16, False, True, False, None, 1.0), (1, 16384, "rms", torch.float32, False, True, False, 1, 1.0),
]


def inputs(m, k, dtype, branch, gamma, beta, groups, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*s, std=1.0, mean=0.0):
        return torch.randn(s, generator=g, device=DEV) * std + mean

    x, b = normal(m, k, std=2.0, mean=0.3).to(dtype), normal(m, k).to(BF16)
    vec = [normal(k, std=0.2, mean=c).to(BF16) if w else None for w, c in ((gamma, 1.0), (beta, 0.0), (branch, 1.0))]
    mod = [None] * 3 if groups is None else list(normal(groups, 3 * k, std=0.4).to(BF16).chunk(3, dim=1))
    return x, b, vec, mod


@pytest.mark.parametrize("m,k,kind,dtype,branch,gamma,beta,groups,alpha", CASES)
def test_against_formula(w8a8, m, k, kind, dtype, branch, gamma, beta, groups, alpha):
    x, b, (ga, be, bg), (gate, scale, shift) = inputs(m, k, dtype, branch, gamma, beta, groups, m + k)
    rpg = 0 if groups is None else -(-m // groups)
    kw = dict(gamma=ga, beta=be, eps=1e-5, kind=w8a8.LAYER_NORM if kind == "layer" else w8a8.RMS_NORM, alpha=alpha,
              gate=gate, branch_gamma=bg, mod_scale=scale, mod_shift=shift, rows_per_group=rpg)
    x0 = x.clone()
    h, img, sx, xq, y = w8a8.residual_norm_quant(x, b, codes=True, y=True, **kw)
    assert torch.equal(x, x0) and h.dtype == dtype
    eh, dh, ey, dy = exact(x, b, ga, be, 1e-5, kind == "layer", alpha, gate, bg, scale, shift, rpg)
    tiny = 1e-30
    assert ((h.double() - eh).abs() <= half_step(dtype) * eh.abs() + dh * 1.01 + tiny).all()
    assert ((y.double() - ey).abs() <= half_step(BF16) * ey.abs() + dy * 1.01 + tiny).all()
    top = ey.abs().amax(1)
    ds = dy.amax(1) / 127 + 2 * U * top / 127
    assert ((sx.double() - top / 127).abs() <= ds + tiny).all()
    s = sx.double()[:, None]
    off = (xq.double() * s - ey).abs()
    assert (off <= s * (0.5 + 127 * 4 * U) + dy * 1.01 + tiny).all()
    assert (xq.abs().amax(1) == 127).all()
    assert torch.equal(img.float(), xq.float())
    # each output by itself: the same bits; in place on the residual stream
    only = w8a8.residual_norm_quant(x, b, image=True, h_out=x, **kw)
    assert only[0].data_ptr() == x.data_ptr() and torch.equal(x, h)
    assert torch.equal(only[1], img) and torch.equal(only[2], sx) and only[3] is None and only[4] is None
    x.copy_(x0)
    only = w8a8.residual_norm_quant(x, b, image=False, y=True, **kw)
    assert torch.equal(only[4], y) and only[1] is None and only[2] is None
    only = w8a8.residual_norm_quant(x, b, image=False, codes=True, **kw)
    assert torch.equal(only[3], xq) and torch.equal(only[2], sx)


def test_zero_rows_and_small_scales(w8a8):
    """A row of zeros has scale 0 and codes 0; values so small that the scale
    is subnormal still give codes."""
    x = torch.zeros(3, 64, device=DEV)
    b = torch.zeros(3, 64, dtype=BF16, device=DEV)
    shift = torch.zeros(3, 64, dtype=BF16, device=DEV)
    shift[1] = 1e-37
    shift[1, 5] = 2e-37
    shift[2] = torch.linspace(-1, 1, 64, device=DEV).to(BF16)
    _, img, sx, xq, _ = w8a8.residual_norm_quant(x, b, mod_shift=shift, rows_per_group=1, codes=True)
    assert sx[0] == 0 and (xq[0] == 0).all() and (img[0] == 0).all() and not torch.signbit(img[0]).any()
    want = torch.round(shift[1].double() / sx[1].double())
    assert 0 < float(sx[1]) < 2.0 ** -126 and (xq[1].double() - want).abs().max() == 0
    assert xq[2, 0] == -127 and xq[2, 63] == 127


def test_large_mean_is_taken_off_first(w8a8):
    """LayerNorm of rows whose mean is 1000 times their spread."""
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(6, 3000, generator=g, device=DEV) + 1000
    b = torch.randn(6, 3000, generator=g, device=DEV).to(BF16)
    h, _, _, _, y = w8a8.residual_norm_quant(x, b, kind=w8a8.LAYER_NORM, image=False, y=True)
    eh, dh, ey, dy = exact(x, b, None, None, 1e-6, True, 1.0, None, None, None, None, 0)
    assert ((y.double() - ey).abs() <= half_step(BF16) * ey.abs() + dy * 1.01).all()


def test_follows_the_linear(w8a8):
    """Its image and scales go into the W8A8 GEMM as they are."""
    x, b, (ga, _, _), _ = inputs(300, 512, BF16, False, True, False, None, 9)
    w = (torch.randn(256, 512, device=DEV) * 0.05).to(BF16)
    wq, sw = w8a8.quantize_weight(w)
    _, img, sx, xq, _ = w8a8.residual_norm_quant(x, b, gamma=ga, codes=True)
    assert torch.equal(w8a8.gemm_postscale_images(img, sx, w8a8.pack_weight(wq), sw),
                       w8a8.gemm_postscale(xq, sx, wq, sw))


def test_refusals(w8a8):
    x = torch.zeros(4, 64, dtype=BF16, device=DEV)
    v = torch.zeros(64, dtype=BF16, device=DEV)
    g2 = torch.zeros(2, 64, dtype=BF16, device=DEV)
    wide = torch.zeros(2, 128, dtype=BF16, device=DEV)
    f = w8a8.residual_norm_quant
    cases = [
        (TypeError, lambda: f(x.half(), x)), (TypeError, lambda: f(x, x.float())), (ValueError, lambda: f(x, x[:2])),
        (ValueError, lambda: f(x.t(), x.t())), (ValueError, lambda: f(x, x, gamma=v[:32])),
        (TypeError, lambda: f(x, x, gamma=v.float())), (ValueError, lambda: f(x, x, gate=g2)),
        (ValueError, lambda: f(x, x, gate=g2, rows_per_group=1)),
        (ValueError, lambda: f(x, x, gate=g2, mod_scale=wide[:, :64], rows_per_group=2)),
        (ValueError, lambda: f(x, x, gate=g2, mod_scale=v, rows_per_group=2)),
        (TypeError, lambda: f(x, x, gate=g2.float(), rows_per_group=2)), (ValueError, lambda: f(x, x, h_out=x[:2])),
        (w8a8.W8A8Error, lambda: f(x, x, eps=-1.0)), (w8a8.W8A8Error, lambda: f(x, x, kind=3)),
        (w8a8.W8A8Error, lambda: f(x[:, :12].contiguous(), x[:, :12].contiguous())),
    ]
    for err, call in cases:
        with pytest.raises(err):
            call()
    assert f(x[:0], x[:0])[0].shape == (0, 64)


@pytest.mark.parametrize("m,k,kind,dtype,branch,gamma,beta,groups,alpha", [
    (2000, 4096, "layer", torch.float32, True, True, True, 7, 1.0), (1000, 5120, "rms", torch.float32, False, True, False, 1000, 1.0),
    (1900, 8184, "layer", torch.float32, False, False, False, 3, -0.5), (913, 2056, "rms", torch.float32, True, False, True, None, 1.0),
    (1300, 2048, "rms", BF16, False, True, False, 650, 1.0),
])
def test_groups_along_many_rows(w8a8, m, k, kind, dtype, branch, gamma, beta, groups, alpha):
    """More rows than are worked on at once, so that each place for a row meets several groups."""
    test_against_formula(w8a8, m, k, kind, dtype, branch, gamma, beta, groups, alpha)
