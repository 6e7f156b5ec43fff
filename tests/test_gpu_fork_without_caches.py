"""The C entry point of forks without caches or pages: W8A8_OK, and nothing is written."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n_caches,pages", [(0, 5), (1, 0), (0, 0)])
def test_nothing_happens(w8a8, n_caches, pages):
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    cache = torch.randn(5, 16, 64, device="cuda").to(torch.bfloat16)
    table, lens = ints(*range(12)).view(4, 3), ints(20, 7, 3, 0)
    src, dst, new = ints(0, 1), ints(2, 3), ints(3, 4)
    keep = [t.clone() for t in (cache, table, lens)]
    at = lambda t: ctypes.c_void_p(t.data_ptr())
    status = w8a8.lib().w8a8_fork_sequences(
        (ctypes.c_void_p * 1)(cache.data_ptr()), (ctypes.c_int64 * 1)(16 * 64 * 2), n_caches, pages, 16 * 64 * 2, 16,
        at(table), 4, 3, 3, at(lens), at(src), at(dst), at(new), 2,
        ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert status == 0
    assert all(torch.equal(a, b) for a, b in zip(keep, (cache, table, lens)))
