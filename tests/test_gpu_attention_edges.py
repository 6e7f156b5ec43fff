"""Attention without keys."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, FP16 = torch.bfloat16, torch.float16


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n,hq,hk,d,dtype", [(1, 8, 2, 128, BF16), (17, 4, 4, 64, FP16), (200, 8, 2, 128, BF16),
                                             (300, 6, 1, 40, FP16)])
def test_no_keys_at_all(w8a8, n, hq, hk, d, dtype, causal):
    """K and V of no rows: every query sees nothing, however many there are."""
    q = torch.randn(n, hq, d, device=DEV).to(dtype)
    k = torch.empty(0, hk, d, dtype=dtype, device=DEV)
    cu_q = torch.tensor([0, n // 2, n], dtype=torch.int32, device=DEV)
    cu_k = torch.zeros(3, dtype=torch.int32, device=DEV)
    for kw in (dict(), dict(cu_q=cu_q, cu_k=cu_k), dict(cu_q=cu_q, k_lens=cu_k[:2])):
        o, lse = w8a8.attention(q, k, torch.empty_like(k), causal=causal, lse=True, **kw)
        assert (o == 0).all() and (lse == -math.inf).all()
    assert w8a8.get_device_error() == (0, 0)
