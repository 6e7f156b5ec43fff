"""NaN and infinities reach the scale of their row, whatever is asked for, and
no other row."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("where", ["x", "b", "shift", "gamma", "gate"])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("m,k,dtype", [(4, 512, BF16), (3000, 1024, BF16), (1300, 2048, torch.float32)])
@pytest.mark.parametrize("options", [False, True])
def test_shows_in_the_scale(w8a8, m, k, dtype, kind, where, bad, options):
    """A row whose y is not finite somewhere has a scale that is not finite, so
    that the Linear after it does not give finite numbers."""
    if not options and where in ("shift", "gate"):
        pytest.skip("an option")
    g = torch.Generator(device=DEV).manual_seed(k)
    x = torch.randn(m, k, generator=g, device=DEV).to(dtype)
    b = torch.randn(m, k, generator=g, device=DEV).to(BF16)
    gamma = torch.ones(k, dtype=BF16, device=DEV)
    shift = torch.zeros(2, k, dtype=BF16, device=DEV)
    gate = torch.ones(2, k, dtype=BF16, device=DEV)
    rows = torch.zeros(m, dtype=torch.bool, device=DEV)
    half = -(-m // 2)
    if where in ("x", "b"):
        (x if where == "x" else b)[m // 3, k // 2] = bad
        rows[m // 3] = True
    elif where == "gamma":
        gamma[7] = bad
        rows[:] = True
    else:
        (shift if where == "shift" else gate)[1, k - 1] = bad
        rows[half:] = True
    kw = dict(gamma=gamma, kind=w8a8.LAYER_NORM if kind == "layer" else w8a8.RMS_NORM)
    if options:
        kw.update(mod_shift=shift, gate=gate, rows_per_group=half)
    _, img, sx, xq, _ = w8a8.residual_norm_quant(x, b, codes=True, **kw)
    assert not torch.isfinite(sx[rows]).any()
    assert torch.isfinite(sx[~rows]).all() and torch.isfinite(img[~rows]).all()
    w, sw = w8a8.quantize_weight(torch.randn(16, k, generator=g, device=DEV).to(BF16))
    y = w8a8.gemm_postscale(xq, sx, w, sw)
    assert not torch.isfinite(y[rows]).any() and torch.isfinite(y[~rows]).all()
    assert w8a8.get_device_error() == (0, 0)
