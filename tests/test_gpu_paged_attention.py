"""Attention over pages against softmax(scale Q K^T) V in 64 bits, with the
tolerance that test_gpu_attention derives (the same products, weights and sums)."""
import math

import pytest
import torch

from test_gpu_attention import check, starts

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, FP16 = torch.bfloat16, torch.float16


class Paged:
    """Random caches in pages in any order; rows that are no key hold NaN, and
    entries of the table past the last page are no pages."""

    def __init__(self, lens, page, hk, d, dtype, seed, layout="token", spare=3):
        g = torch.Generator(device=DEV).manual_seed(seed)
        used = [-(-m // page) for m in lens]
        pages = sum(used) + spare
        shape = (pages, page, hk, d)
        if layout == "token":
            kv = [torch.full(shape, math.nan, dtype=dtype, device=DEV) for _ in range(2)]
        elif layout == "head":  # every head's rows of a page together
            kv = [torch.full((pages, hk, page, d), math.nan, dtype=dtype, device=DEV).transpose(1, 2) for _ in range(2)]
        else:  # K and V of a page side by side, in a wider row
            both = torch.full((pages, 2, page, hk, d + 8), math.nan, dtype=dtype, device=DEV)
            kv = [both[:, 0, :, :, :d], both[:, 1, :, :, :d]]
        self.k_pages, self.v_pages = kv
        self.table = torch.full((len(lens), max(used, default=0) + 2), -7, dtype=torch.int32, device=DEV)
        self.table[:, 1::2] = 1 << 30
        order = torch.randperm(pages, generator=g, device=DEV)
        self.k, self.v, at = [], [], 0
        for b, m in enumerate(lens):
            mine = order[at:at + used[b]]
            at += used[b]
            self.table[b, :used[b]] = mine.to(torch.int32)
            i = torch.arange(m, device=DEV)
            for cache, parts in zip(kv, (self.k, self.v)):
                x = torch.randn(m, hk, d, generator=g, device=DEV).to(dtype)
                cache[mine[i // page], i % page] = x
                parts.append(x)
        self.k_lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
        self.lens = lens

    def flat(self):
        return torch.cat(self.k), torch.cat(self.v)


def queries(tokens, hq, d, dtype, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(tokens, hq + 2, d, generator=g, device=DEV).to(dtype)[:, 1:hq + 1]


CASES = [
    # (queries, keys), page, heads, dim
    ([1], [1], 16, 1, 1, 64, BF16, "token"),
    ([1, 1, 1, 1], [5, 63, 64, 65], 16, 32, 8, 128, BF16, "token"),
    ([1, 1, 1, 1], [300, 0, 129, 2], 24, 5, 1, 64, FP16, "head"),
    ([1], [40000], 64, 8, 1, 128, BF16, "token"),
    ([2, 2, 2], [9000, 17, 5000], 48, 40, 8, 128, BF16, "pair"),
    ([3] * 40, [777] * 40, 8, 28, 4, 128, FP16, "token"),
    ([16, 16], [20000, 16], 128, 4, 4, 128, BF16, "head"),
    ([30, 31], [512, 100], 256, 20, 4, 64, BF16, "pair"),
    ([64], [5000], 64, 40, 8, 128, BF16, "token"),
    ([200], [3000], 40, 8, 8, 128, FP16, "token"),
    ([513, 130], [513, 130], 16, 12, 4, 96, FP16, "token"),
    ([700], [4500], 1000, 20, 1, 128, FP16, "head"),
    ([5, 1, 64, 200, 1, 0], [300, 1, 64, 1000, 4000, 9], 32, 8, 2, 128, BF16, "token"),
    ([260, 1, 1, 1, 33], [4100, 9, 700, 1, 33], 16, 5, 1, 128, BF16, "pair"),
    ([300, 4, 129, 1], [20, 0, 128, 0], 16, 4, 2, 128, BF16, "token"),   # more queries than keys
    ([7, 0, 3], [0, 50, 3], 16, 16, 2, 64, FP16, "token"),
    ([1] * 70 + [40, 3], [(i * 131) % 900 for i in range(70)] + [640, 3], 64, 12, 1, 40, BF16, "token"),
    ([100, 2], [1000, 77], 80, 130, 1, 8, BF16, "token"),                # a group of more heads than a tile's rows
    ([9, 17, 128], [400, 2000, 150], 16, 34, 2, 120, BF16, "token"),     # groups that do not divide the tile's rows
    ([1537], [1537], 64, 2, 1, 128, BF16, "token"),
    ([4, 2, 6], [300, 64, 120], 16, 40, 8, 128, BF16, "head"),           # two MMA tiles of rows, few keys
    ([31, 0, 7], [200, 5, 3], 8, 4, 4, 72, FP16, "pair"),
    ([3, 9, 1], [700, 40, 1], 32, 100, 1, 64, BF16, "token"),            # one query a tile, rows to spare
    ([3, 1, 2], [700, 40, 129], 32, 256, 2, 128, FP16, "head"),          # and none to spare
    ([40, 1, 3], [900, 2000, 3], 24, 14, 7, 48, BF16, "token"),          # seven KV heads
    ([40, 1, 3], [900, 2000, 3], 24, 11, 11, 128, BF16, "pair"),         # a prime number of them
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n,m,page,hq,hk,d,dtype,layout", CASES)
def test_paged_attention(w8a8, n, m, page, hq, hk, d, dtype, layout, causal):
    c = Paged(m, page, hk, d, dtype, 1 + page + hq, layout)
    q = queries(sum(n), hq, d, dtype, 2 + d)
    k, v = c.flat()
    results = []
    for most in (None, max(n)):
        o, lse = w8a8.paged_attention(q, c.k_pages, c.v_pages, c.table, c.k_lens, cu_q=starts(n), max_queries=most,
                                      causal=causal, lse=True)
        check(o, lse, q, k, v, n, m, causal, d ** -0.5)
        results.append((o, lse))
    if len(set(n)) == 1:  # equal parts need no bounds
        o, lse = w8a8.paged_attention(q, c.k_pages, c.v_pages, c.table, c.k_lens, causal=causal, lse=True)
        check(o, lse, q, k, v, n, m, causal, d ** -0.5)
    assert w8a8.get_device_error() == (0, 0)


@pytest.mark.parametrize("n,m,page,hq,hk,d,dtype", [
    ([300], [9000], 48, 8, 8, 128, BF16), ([260, 150], [8700, 9999], 64, 32, 8, 128, FP16), ([513], [17000], 16, 16, 8, 64, BF16),
    ([70], [16500], 256, 24, 4, 128, BF16), ([1300], [8500], 40, 8, 8, 128, BF16)])
def test_many_keys_and_rows(w8a8, n, m, page, hq, hk, d, dtype):
    """Caches that fill a good part of L2 (where pieces do not begin with their first key
    tile), with values that are not finite among keys that only the last rows see."""
    c = Paged(m, page, hk, d, dtype, 81)
    q = queries(sum(n), hq, d, dtype, 82)
    call = lambda: w8a8.paged_attention(q, c.k_pages, c.v_pages, c.table, c.k_lens, cu_q=starts(n), lse=True)
    o, lse = call()
    check(o, lse, q, *c.flat(), n, m, True, d ** -0.5)
    for _ in range(5):
        again = call()
        assert torch.equal(again[0], o) and torch.equal(again[1], lse)
    at = m[0] - n[0] // 2
    c.v_pages[int(c.table[0, at // page]), at % page] = math.inf
    o, lse = call()
    first = n[0] - n[0] // 2
    check(o[:first], lse[:first], q[:first], c.k[0][:at], c.v[0][:at], [first], [at], True, d ** -0.5)
    assert not torch.isfinite(o[first:n[0]]).any()
    for b in range(1, len(n)):
        check(o[n[0]:], lse[n[0]:], q[n[0]:], c.k[b], c.v[b], n[1:], m[1:], True, d ** -0.5)
    assert w8a8.get_device_error() == (0, 0)


def test_the_most_queries_need_not_be_true(w8a8):
    n, m = [1, 90, 5], [500, 600, 700]
    c = Paged(m, 32, 2, 64, BF16, 3)
    q = queries(sum(n), 8, 64, BF16, 4)
    for most in (1, 4, 1000, 1 << 40):
        o, lse = w8a8.paged_attention(q, c.k_pages, c.v_pages, c.table, c.k_lens, cu_q=starts(n), max_queries=most,
                                      lse=True)
        check(o, lse, q, *c.flat(), n, m, True, 64 ** -0.5)


@pytest.mark.parametrize("most", [None, 60])
def test_few_rows_that_are_all_of_one_sequence(w8a8, most):
    """As many rows as sequences, which single tokens would be."""
    n, m = [0, 60] + [0] * 58, [40, 700] + [9] * 58
    c = Paged(m, 16, 2, 64, BF16, 121)
    q = queries(sum(n), 8, 64, BF16, 122)
    o, lse = w8a8.paged_attention(q, c.k_pages, c.v_pages, c.table, c.k_lens, cu_q=starts(n), max_queries=most, lse=True)
    check(o, lse, q, *c.flat(), n, m, True, 0.125)


@pytest.mark.parametrize("n", [1, 7, 150])
def test_pages_outside_the_cache_are_zeros(w8a8, n):
    m, page, d = 900, 48, 128
    c = Paged([m], page, 2, d, BF16, 8)
    q = queries(n, 8, d, BF16, 9)
    for column, value in ((0, -1), (5, c.k_pages.shape[0]), (9, (1 << 31) - 1), (18, -(1 << 31))):
        c.table[0, column] = value
        c.k[0][column * page:(column + 1) * page] = 0
        c.v[0][column * page:(column + 1) * page] = 0
    o, lse = w8a8.paged_attention(q, c.k_pages, c.v_pages, c.table, c.k_lens, lse=True)
    check(o, lse, q, *c.flat(), [n], [m], True, d ** -0.5)


@pytest.mark.parametrize("n", [1, 33, 300])
def test_lengths_and_bounds_are_clamped(w8a8, n):
    c = Paged([250, 256], 64, 2, 64, BF16, 5, spare=0)
    table = c.table[:, :4].contiguous()
    q = queries(2 * n, 4, 64, BF16, 6)
    for lens, want in (([-5, 1 << 30], [0, 256]), ([250, 257], [250, 256])):
        k_lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
        o, lse = w8a8.paged_attention(q, c.k_pages, c.v_pages, table, k_lens, lse=True)
        k, v = (torch.cat([x[0][:want[0]], x[1]]) for x in (c.k, c.v))
        check(o, lse, q, k, v, [n, n], want, True, 0.125)
    # the first sequence's queries start before the tensor, the second's end behind it
    cu = torch.tensor([-9, n, 1 << 30], dtype=torch.int32, device=DEV)
    o, lse = w8a8.paged_attention(q, c.k_pages, c.v_pages, table, c.k_lens, cu_q=cu, lse=True)
    check(o, lse, q, *c.flat(), [n, n], [250, 256], True, 0.125)


def test_no_keys_at_all(w8a8):
    q = queries(40, 4, 64, BF16, 6)
    pages = torch.empty(0, 16, 2, 64, dtype=BF16, device=DEV)
    lens = torch.tensor([7, 9], dtype=torch.int32, device=DEV)
    table = torch.zeros(2, 3, dtype=torch.int32, device=DEV)
    some = torch.ones(4, 16, 2, 64, dtype=BF16, device=DEV)
    for kv, t in ((pages, table), (some, table[:, :0])):
        o, lse = w8a8.paged_attention(q, kv, kv, t, lens, lse=True)
        assert (o == 0).all() and (lse == -math.inf).all()
    assert w8a8.paged_attention(q[:0], some, some, table, lens).shape == (0, 4, 64)
    none = torch.empty(0, 3, dtype=torch.int32, device=DEV)
    assert w8a8.paged_attention(q[:0], some, some, none, lens[:0]).shape == (0, 4, 64)


@pytest.mark.parametrize("n", [1, 20, 290])
def test_rows_of_no_sequence_stay(w8a8, n):
    c = Paged([300, 310], 16, 2, 128, FP16, 11)
    q = queries(2 * n + 9, 8, 128, FP16, 12)
    out = torch.full((2 * n + 9, 8, 128), 7.0, dtype=FP16, device=DEV)
    cu = torch.tensor([4, 4 + n, 4 + 2 * n], dtype=torch.int32, device=DEV)
    r, lse = w8a8.paged_attention(q, c.k_pages, c.v_pages, c.table, c.k_lens, cu_q=cu, out=out, lse=True)
    assert r is out and (out[:4] == 7).all() and (out[4 + 2 * n:] == 7).all()
    check(out[4:-5], lse[4:-5], q[4:-5], *c.flat(), [n, n], [300, 310], True, 128 ** -0.5)


@pytest.mark.parametrize("n", [1, 40, 333])
def test_what_a_row_does_not_see(w8a8, n):
    """Infinities and NaN in V of keys that only later queries see, and K as well:
    rows before do not change; rows that see them are not finite."""
    m, d = n + 700, 128
    c = Paged([m], 32, 2, d, BF16, 21)
    q = queries(n, 8, d, BF16, 22)
    for at, value in ((m - 1, math.nan), (m - n + n // 2, math.inf)):
        page, row = int(c.table[0, at // 32]), at % 32
        for cache in (c.v_pages, c.k_pages):
            keep = cache[page, row].clone()
            cache[page, row] = value
            o, lse = w8a8.paged_attention(q, c.k_pages, c.v_pages, c.table, c.k_lens, lse=True)
            first = at - (m - n)
            check(o[:first], lse[:first], q[:first], c.k[0][:at], c.v[0][:at], [first], [at], True, d ** -0.5)
            if cache is c.v_pages:
                assert not torch.isfinite(o[first:]).any()
            cache[page, row] = keep


def test_sinks_and_moving_maxima(w8a8):
    """Scores that grow along the keys, and one key that takes nearly all weight in the middle of a long cache."""
    for dtype in (BF16, FP16):
        for n in (1, 3, 130):
            m, d = 9000, 64
            c = Paged([m], 64, 1, d, dtype, 31)
            q = queries(n, 4, d, dtype, 32).abs() + 0.1
            grow = torch.linspace(-3, 3, m, device=DEV)[:, None, None]
            k = (c.k[0].float() * 0.1 + grow).to(dtype)
            k[4321] = 6.0
            i = torch.arange(m, device=DEV)
            c.k_pages[c.table[0].long()[i // 64], i % 64] = k
            o, lse = w8a8.paged_attention(q, c.k_pages, c.v_pages, c.table, c.k_lens, lse=True, scale=0.3)
            check(o, lse, q, k, c.v[0], [n], [m], True, 0.3)


def test_the_same_bits_every_time(w8a8):
    n, m = [1, 300, 7, 1, 50], [5000, 4000, 900, 30, 8000]
    c = Paged(m, 16, 4, 128, BF16, 41)
    q = queries(sum(n), 16, 128, BF16, 42)
    call = lambda **kw: w8a8.paged_attention(q, c.k_pages, c.v_pages, c.table, c.k_lens, cu_q=starts(n), lse=True, **kw)
    first = call()
    for _ in range(20):
        again = call()
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])
    ws = w8a8.paged_attention_workspace()
    again = call(workspace=ws)
    assert torch.equal(again[0], first[0])
    # a workspace full of anything behind its counters
    ws[w8a8.lib().w8a8_attention_workspace_zeroed():] = 0xFF
    assert torch.equal(call(workspace=ws)[0], first[0])


def test_captured_calls_and_streams(w8a8):
    """Two captured graphs, replayed in turn and beside eager calls on two streams, with lengths that change between replays."""
    n, cap = [1, 60, 1], 40
    c = Paged([900, 700, 1100], 32, 2, 128, BF16, 51)
    q = queries(sum(n), 8, 128, BF16, 52)
    cu = starts(n)
    side = torch.cuda.Stream()
    call = lambda: w8a8.paged_attention(q, c.k_pages, c.v_pages, c.table, c.k_lens, cu_q=cu)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call())
        graphs.append(g)
    for step in range(4):
        c.k_lens.copy_(torch.tensor([900 - step * 100, 700 - step * 90, 1100 - step], dtype=torch.int32))
        want = call()
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graphs[0].replay()
        graphs[1].replay()
        with torch.cuda.stream(side):
            other = call()
        torch.cuda.synchronize()
        for o in (*outs, other):
            assert torch.equal(o, want)
    assert w8a8.get_device_error() == (0, 0)


def test_offsets_past_32_bits(w8a8):
    """Pages whose rows lie past 2^32 bytes and 2^31 elements of the cache."""
    page, hk, d = 64, 8, 128
    pages = (5 << 30) // (page * hk * d * 2) + 1
    k_pages = torch.zeros(pages, page, hk, d, dtype=BF16, device=DEV)
    v_pages = torch.zeros_like(k_pages)
    g = torch.Generator(device=DEV).manual_seed(3)
    far = torch.tensor([pages - 1, 3, pages - 2, pages // 2, pages - 9], device=DEV)
    m = 5 * page - 7
    k, v = (torch.randn(m, hk, d, generator=g, device=DEV).to(BF16) for _ in range(2))
    i = torch.arange(m, device=DEV)
    k_pages[far[i // page], i % page] = k
    v_pages[far[i // page], i % page] = v
    table = far[None].to(torch.int32)
    for n in (1, 100):
        q = queries(n, 32, d, BF16, n)
        o, lse = w8a8.paged_attention(q, k_pages, v_pages, table, torch.tensor([m], dtype=torch.int32, device=DEV), lse=True)
        check(o, lse, q, k, v, [n], [m], True, d ** -0.5)


def test_a_table_shared_by_all(w8a8):
    """One row of pages for every sequence (a broadcast table), at different lengths."""
    c = Paged([600], 16, 2, 64, BF16, 61)
    lens = [600, 1, 333, 64]
    q = queries(4, 4, 64, BF16, 62)
    o, lse = w8a8.paged_attention(q, c.k_pages, c.v_pages, c.table.expand(4, -1),
                                  torch.tensor(lens, dtype=torch.int32, device=DEV), lse=True)
    k, v = (torch.cat([x[0][:m] for m in lens]) for x in (c.k, c.v))
    check(o, lse, q, k, v, [1] * 4, lens, True, 0.125)


def test_thousands_of_sequences(w8a8):
    """More sequences than a warp counts at once, two of them with many queries, without a word about it."""
    n = [1] * 3000
    n[0], n[1700], n[2999] = 37, 150, 2
    m = [q + (i * 37) % 150 for i, q in enumerate(n)]
    c = Paged(m, 16, 1, 64, BF16, 91)
    q = queries(sum(n), 4, 64, BF16, 92)
    o, lse = w8a8.paged_attention(q, c.k_pages, c.v_pages, c.table, c.k_lens, cu_q=starts(n), lse=True)
    k, v = c.flat()
    cq, ck = starts(n).tolist(), starts(m).tolist()
    for b in [0, 1, 31, 32, 33, 1699, 1700, 1701, 2047, 2998, 2999] + list(range(100, 3000, 97)):
        rows, keys = slice(cq[b], cq[b + 1]), slice(ck[b], ck[b + 1])
        check(o[rows], lse[rows], q[rows], k[keys], v[keys], [n[b]], [m[b]], True, 0.125)
    assert torch.isfinite(o).all()
    alone = [i for i, x in enumerate(n) if x == 1]
    rows = starts(n).long()[:-1][torch.tensor(alone, device=DEV)]
    o1 = w8a8.paged_attention(q[rows], c.k_pages, c.v_pages, c.table[alone], c.k_lens[alone], max_queries=1)
    assert (o1.double() - o[rows].double()).abs().max() <= 4 * 2.0 ** -8 * 4


@pytest.mark.parametrize("n", [1, 45])
def test_a_million_keys(w8a8, n):
    """Pages that come again and again: what the same keys give once."""
    c = Paged([256], 64, 2, 64, BF16, 95)
    times = 4096
    q = queries(n, 16, 64, BF16, 96)
    table = c.table[:, :4].repeat(1, times)
    lens = torch.tensor([256 * times], dtype=torch.int32, device=DEV)
    o, lse = w8a8.paged_attention(q, c.k_pages, c.v_pages, table, lens, causal=False, lse=True)
    want, lse1 = w8a8.paged_attention(q, c.k_pages, c.v_pages, c.table, c.k_lens, causal=False, lse=True)
    # sums of 2^20 terms in binary32, in parts: at most 2^-24 of the total for each of the 2^20 / 16 additions of one lane
    tol = 2.0 ** -8 * (want.double().abs() + 2.0 ** -4) + 2.0 ** -8 * c.v[0].double().abs().mean()
    assert ((o.double() - want.double()).abs() <= tol).all()
    assert (lse - lse1 - math.log(times)).abs().max() <= 2.0 ** -8


def test_two_streams_at_once(w8a8):
    n, m = [120, 1, 1, 30], [3000, 2500, 40, 900]
    sides, want, cases = [torch.cuda.Stream() for _ in range(2)], [], []
    for i in range(2):
        c = Paged(m, 16, 4, 128, BF16, 101 + i)
        cases.append((queries(sum(n), 16, 128, BF16, 103 + i), c.k_pages, c.v_pages, c.table, c.k_lens, starts(n)))
        want.append(w8a8.paged_attention(*cases[i]))
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(30):
        for i in range(2):
            with torch.cuda.stream(sides[i]):
                got[i].append(w8a8.paged_attention(*cases[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for o in got[i]:
            assert torch.equal(o, want[i])
    assert w8a8.get_device_error() == (0, 0)


def test_one_query_for_all_sequences(w8a8):
    """A broadcast Q: the same query row for every sequence."""
    c = Paged([100, 7, 300], 16, 2, 64, BF16, 111)
    q = queries(1, 8, 64, BF16, 112)
    o, lse = w8a8.paged_attention(q.expand(3, -1, -1), c.k_pages, c.v_pages, c.table, c.k_lens, lse=True)
    check(o, lse, q.repeat(3, 1, 1), *c.flat(), [1, 1, 1], [100, 7, 300], True, 0.125)


def test_refusals(w8a8):
    c = Paged([60], 16, 2, 64, BF16, 71)
    q = queries(2, 4, 64, BF16, 72)
    call = lambda **kw: w8a8.paged_attention(**{**dict(Q=q, k_pages=c.k_pages, v_pages=c.v_pages, page_table=c.table,
                                                       k_lens=c.k_lens), **kw})
    for match, kw in (("out must have the shape", dict(out=q[:1].clone())), ("max_queries", dict(max_queries=-1)),
                      ("workspace", dict(workspace=torch.empty(4, 4, dtype=torch.uint8, device=DEV).t()[1:]))):
        with pytest.raises(ValueError, match=match):
            call(**kw)
    for kw in (dict(workspace=torch.zeros(1 << 20, dtype=torch.uint8, device=DEV)), dict(scale=0.0),
               dict(k_pages=c.k_pages[:1].expand(4, -1, -1, -1), v_pages=c.v_pages[:1].expand(4, -1, -1, -1))):
        with pytest.raises(w8a8.W8A8Error):
            call(**kw)
