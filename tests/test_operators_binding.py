"""Refusals of tensors by the operators' Python calls (CPU tensors: nothing
gets as far as the library)."""
import pytest
import torch


@pytest.fixture(scope="module")
def w():
    from w8a8_int8_linear_gb300 import build as b
    b.build()
    import w8a8_int8_linear_gb300 as w
    return w


X = torch.zeros(4, 2, 64, dtype=torch.bfloat16)


@pytest.mark.parametrize("error,match,call", [
    (TypeError, "Q must be a torch.Tensor", lambda w: w.attention([1], X, X)),
    (TypeError, "Q must be torch.bfloat16 or torch.float16, got torch.float32", lambda w: w.attention(X.float(), X, X)),
    (ValueError, "Q must be a CUDA tensor", lambda w: w.attention(X, X, X)),
    (TypeError, "unexpected keyword", lambda w: w.attention(X, X, X, mask=X)),
    (ValueError, "layout must be 'half' or 'interleaved'", lambda w: w.rotary(X, X, X, X, layout="both")),
    (ValueError, "Q must be a CUDA tensor", lambda w: w.rotary(X, None, X, X)),
    (ValueError, "Q must be a CUDA tensor", lambda w: w.rotary_append(X, X, X, X, X, X, X, X)),
    (TypeError, "Q must be a torch.Tensor", lambda w: w.rotary_append(None, X, X, X, X, X, X, X)),
    (ValueError, r"X must be a \[rows, width\] tensor", lambda w: w.residual_norm_quant(X, X)),
    (TypeError, "X must be torch.bfloat16 or torch.float32", lambda w: w.residual_norm_quant(X[0].half(), X[0])),
    (ValueError, r"X must be a dense CUDA tensor of shape \[2, 64\]", lambda w: w.residual_norm_quant(X[0], X[0])),
    (TypeError, "", lambda w: w.residual_norm_quant(X[0], X[0], rows_per_group="a")),
])
def test_refusals(w, error, match, call):
    with pytest.raises(error, match=match):
        call(w)
