"""What the operators write in place is known to autograd as written."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16


def calls(w):
    q = torch.randn(4, 2, 32, device=DEV).to(BF16)
    rows, branch = torch.randn(2, 4, 64, device=DEV).to(BF16)
    pos, f = torch.arange(4, device=DEV), w.rotary_frequencies(32)
    empty = torch.empty_like
    return {
        "attention": ([empty(q)], lambda t: w.attention(q, q, q, out=t[0])),
        "rotary": ([empty(q), empty(q)], lambda t: w.rotary(q, q, pos, f, q_out=t[0], k_out=t[1])),
        "rotary in place": ([q.clone()], lambda t: w.rotary(t[0], None, pos, f, q_out=t[0])),
        "rotary_append": ([empty(q), empty(q), empty(q)],
                          lambda t: w.rotary_append(q, q, q, pos, f, t[0], t[1], pos, q_out=t[2])),
        "residual_norm_quant": ([empty(rows)], lambda t: w.residual_norm_quant(rows, branch, h_out=t[0])),
    }


NAMES = ["attention", "rotary", "rotary in place", "rotary_append", "residual_norm_quant"]


@pytest.mark.parametrize("name", NAMES)
def test_versions(w8a8, name):
    written, call = calls(w8a8)[name]
    before = [t._version for t in written]
    call(written)
    assert all(t._version > v for t, v in zip(written, before))


def test_a_saved_value_that_is_overwritten(w8a8):
    """A backward pass that needs a value which was turned in place says so
    instead of giving a wrong gradient."""
    p = torch.randn(4, 2, 32, device=DEV, requires_grad=True)
    x = torch.randn(4, 2, 32, device=DEV).to(BF16)
    y = (p * x).sum()
    w8a8.rotary(x, None, torch.arange(4, device=DEV), w8a8.rotary_frequencies(32), q_out=x)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


@pytest.mark.parametrize("name", NAMES)
def test_tensors_that_require_a_gradient(w8a8, name):
    written, call = calls(w8a8)[name]
    for i in range(len(written)):
        given = [t.clone().requires_grad_(j == i) for j, t in enumerate(written)]
        with pytest.raises(ValueError, match="requires a gradient"):
            call(given)
        with torch.no_grad():
            call(given)


@pytest.mark.parametrize("name", NAMES)
def test_inference_tensors(w8a8, name):
    """Tensors made in inference mode have no version; they are written there and
    outside of it."""
    with torch.inference_mode():
        written, call = calls(w8a8)[name]
        call(written)
    call(written)
    normal, call = calls(w8a8)[name]
    with torch.inference_mode():
        call(normal)
