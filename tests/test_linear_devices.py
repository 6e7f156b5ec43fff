"""The W8A8 Linear's calls run on the current GPU: tensors on another one are
refused.  The tensors are fake ones, which have a device and no memory."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="fake tensors of any GPU need a machine without one")

BF16, S8, F32 = torch.bfloat16, torch.int8, torch.float32
M, N, K = 300, 256, 512
CODES = dict(Xq=((M, K), S8), sx=((M,), F32), Wq=((N, K), S8), sw=((N,), F32), bias=((N,), BF16), out=((M, N), BF16))
BLOCKS = dict(CODES, sx=((M, K // 128), F32), sw=((N // 128, K // 128), F32))
IMAGES = dict(Ximg=((M, K), BF16), sx=((M,), F32), Wimg=((N, K), BF16), sw=((N,), F32), bias=((N,), BF16),
              out=((M, N), BF16))
LINEAR = dict(X=((M, K), BF16), Wimg=((N, K), BF16), sw=((N,), F32), bias=((N,), BF16), out=((M, N), BF16),
              workspace=((1 << 26,), torch.uint8), sx_out=((M,), F32))
CALLS = {
    "quantize_weight": dict(W=((N, K), BF16)), "quantize_act": dict(X=((M, K), BF16)), "pack_weight": dict(Wq=((N, K), S8)),
    "gemm_postscale": CODES, "gemm_blockwise": BLOCKS, "gemm_postscale_noalloc": CODES, "gemm_postscale_images": IMAGES,
    "gemm_blockwise_images": dict(IMAGES, sx=((M, K // 128), F32), sw=((N // 128, K // 128), F32)),
    "gemm_postscale_s32": dict(Xq=((M, K), S8), Wq=((N, K), S8)),
    "linear_postscale": LINEAR, "linear_postscale_gelu_quant": LINEAR,
    "linear_postscale_codes": {("Wq" if n == "Wimg" else n): ((N, K), S8) if n == "Wimg" else s for n, s in LINEAR.items()},
    "norm_quant": dict(X=((M, K), BF16), gamma=((K,), BF16), beta=((K,), BF16)),
    "gelu_bf16": dict(Y=((M, N), BF16), out=((M, N), BF16)), "stream_floor": dict(src=((M, K), BF16), dst=((M, K), S8)),
}


@pytest.fixture(scope="module")
def w():
    from w8a8_int8_linear_gb300 import build as b
    b.build()
    import w8a8_int8_linear_gb300 as w
    w.lib()
    return w


def test_several_gpus_are_seen(w, monkeypatch):
    monkeypatch.setattr(w, "_several_gpus", False)
    for count in (0, 1, 2, 8):
        monkeypatch.setattr(w, "_lib", None)
        monkeypatch.setattr(torch.cuda, "device_count", lambda: count)
        w.lib()
        assert w._several_gpus == (count > 1)


@pytest.mark.parametrize("call,name", [(c, n) for c, args in CALLS.items() for n in args])
def test_another_gpu(w, monkeypatch, call, name):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(w, "_several_gpus", True)
    with FakeTensorMode():
        args = {n: torch.empty(shape, dtype=dtype, device="cuda:1" if n == name else "cuda:0")
                for n, (shape, dtype) in CALLS[call].items()}
        with pytest.raises(ValueError, match="on cuda:1, but the current device is cuda:0"):
            getattr(w, call)(**args)
