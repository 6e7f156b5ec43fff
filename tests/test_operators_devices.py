"""Refusals of tensors on several GPUs, and of written tensors that require a
gradient, by the operators' Python calls.  The
tensors are fake ones, which have a device and no memory: nothing is launched.
Where there is a GPU, torch makes none of another that is not there."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="fake tensors of any GPU need a machine without one")

BF16, INT, LONG, DOUBLE = torch.bfloat16, torch.int32, torch.int64, torch.float64


@pytest.fixture(scope="module")
def w():
    from w8a8_int8_linear_gb300 import build as b
    b.build()
    import w8a8_int8_linear_gb300 as w
    return w


def on(device, shape, dtype=BF16):
    with FakeTensorMode():
        return torch.empty(shape, dtype=dtype, device=device)


HEADS = (4, 2, 64)
# function, its arguments in order: name -> (shape, type)
CALLS = {
    "attention": dict(Q=(HEADS, BF16), K=(HEADS, BF16), V=(HEADS, BF16), cu_q=((2,), INT), cu_k=((2,), INT),
                      k_lens=((1,), INT), out=(HEADS, BF16), workspace=((1 << 24,), torch.uint8)),
    "rotary": dict(Q=(HEADS, BF16), K=(HEADS, BF16), positions=((4,), LONG), freqs=((16,), DOUBLE), q_out=(HEADS, BF16),
                   k_out=(HEADS, BF16)),
    "rotary_append": dict(Q=(HEADS, BF16), K=(HEADS, BF16), V=(HEADS, BF16), positions=((4,), LONG),
                          freqs=((16,), DOUBLE), k_cache=((9, 2, 64), BF16), v_cache=((9, 2, 64), BF16),
                          slots=((4,), LONG), q_out=(HEADS, BF16)),
    "residual_norm_quant": dict(X=((4, 64), BF16), B=((4, 64), BF16), gamma=((64,), BF16), beta=((64,), BF16),
                                gate=((1, 64), BF16), branch_gamma=((64,), BF16), mod_scale=((1, 64), BF16),
                                mod_shift=((1, 64), BF16), h_out=((4, 64), BF16)),
}


@pytest.mark.parametrize("call,name", [(c, n) for c, args in CALLS.items() for n in list(args)[1:]])
def test_another_gpu(w, call, name):
    first = next(iter(CALLS[call]))
    args = {n: on("cuda:1" if n == name else "cuda:0", *spec) for n, spec in CALLS[call].items()}
    with pytest.raises(ValueError, match=f"{name} is on cuda:1, {first} on cuda:0"):
        getattr(w, call)(**args)


WRITTEN = {"attention": ["out"], "rotary": ["q_out", "k_out"], "rotary_append": ["k_cache", "v_cache", "q_out"],
           "residual_norm_quant": ["h_out"]}


@pytest.mark.parametrize("call,name", [(c, n) for c, names in WRITTEN.items() for n in names])
def test_written_tensors_that_require_a_gradient(w, call, name):
    args = {n: on("cuda:0", *spec) for n, spec in CALLS[call].items()}
    args[name].requires_grad_()
    with pytest.raises(ValueError, match=f"{name} requires a gradient"):
        getattr(w, call)(**args)
