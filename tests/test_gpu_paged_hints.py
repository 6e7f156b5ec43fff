"""Which kernel serves attention over pages when the caller says nothing about the most
queries of a sequence.  The two kernels round differently, so a call's bits tell which it was."""
import pytest
import torch

from test_gpu_attention import check, starts
from test_gpu_paged_attention import Paged, queries

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def calls(w8a8, n, m, hq, hk, d, seed, options):
    c = Paged(m, 16, hk, d, BF16, seed)
    q = queries(sum(n), hq, d, BF16, seed + 1)
    results = [w8a8.paged_attention(q, c.k_pages, c.v_pages, c.table, c.k_lens, cu_q=starts(n), lse=True, **kw)
               for kw in options]
    for o, lse in results:
        check(o, lse, q, *c.flat(), n, m, True, d ** -0.5)
    return [o for o, _ in results]


@pytest.mark.parametrize("n,batch,m,hq,hk", [
    (200, 256, 3000, 40, 8), (60, 60, 3000, 8, 2), (64, 64, 5000, 32, 8), (20, 21, 2000, 12, 4),
    (256, 256, 4000, 4, 4)])
def test_a_chunk_in_a_padded_batch(w8a8, n, batch, m, hq, hk):
    """One chunk among idle sequences, no more rows than sequences: the kernel of many
    queries, as where the caller says how many there are."""
    row = batch // 3
    ns, ms = [0] * batch, [i % 40 for i in range(batch)]
    ns[row], ms[row] = n, m
    unsaid, said, single = calls(w8a8, ns, ms, hq, hk, 128, 7 + n, ({}, dict(max_queries=n), dict(max_queries=1)))
    assert torch.equal(unsaid, said)
    assert not torch.equal(said, single)


@pytest.mark.parametrize("batch,hq,hk", [(12, 40, 8), (16, 32, 8), (5, 48, 4), (40, 4, 4)])
def test_a_few_single_tokens(w8a8, batch, hq, hk):
    """Up to 64 packed rows, a row for each sequence: the kernel of few queries."""
    ms = [900 + 311 * i for i in range(batch)]
    unsaid, said, many = calls(w8a8, [1] * batch, ms, hq, hk, 128, 40 + batch,
                               ({}, dict(max_queries=1), dict(max_queries=batch)))
    assert torch.equal(unsaid, said)
    assert not torch.equal(said, many)
