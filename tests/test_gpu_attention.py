"""Attention against softmax(scale Q K^T) V in 64 bits.

Tolerance, per output element, for u = eps / 2 of the inputs' type (half a
rounding step, relative) and w the exact weights:
  the scores' sums of D products in binary32 are off by at most
  dt = (D + 4) 2^-24 scale sum|q||k|, so each weight by 2 dt relative (its own
  score and the normalizer's), plus 2^-20 for exp2, the binary32 sums of at
  most 2^13 terms in any order and the joins of partial results, plus u for
  its rounding to the inputs' type; fp16 weights below its normal range are
  off by 2^-25 of the row's maximum.  With A = sum w |v|:
    |o - exact| <= (u + 2 dt + 2^-10 u_sum) A + u |exact|,
  where the binary32 sums over m keys contribute m 2^-24 (taken as such)."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, FP16 = torch.bfloat16, torch.float16


def visible(n, m, causal):
    i = torch.arange(n, device=DEV)[:, None]
    j = torch.arange(m, device=DEV)[None, :]
    return (j <= i + m - n) if causal else torch.ones(n, m, dtype=torch.bool, device=DEV)


def exact(q, k, v, causal, scale):
    """q [n, Hq, D], k / v [m, Hk, D] of one sequence -> o, lse, tolerance in 64 bits."""
    n, hq, d = q.shape
    m, hk, _ = k.shape
    dt_ = q.dtype
    q, k, v = (x.double().transpose(0, 1) for x in (q, k, v))
    k, v = (x.repeat_interleave(hq // hk, 0) for x in (k, v))
    see = visible(n, m, causal)
    # what a row does not see does not take part, whatever it holds
    t = torch.matmul(q, k.nan_to_num(0, 0, 0).transpose(1, 2)) * scale
    t = t.masked_fill(~see, -math.inf)
    o = torch.zeros(hq, n, d, dtype=torch.float64, device=DEV)
    lse = torch.full((hq, n), -math.inf, dtype=torch.float64, device=DEV)
    tol = torch.zeros_like(o)
    rows = see.any(1)
    if m and rows.any():
        w = torch.softmax(t[:, rows], -1)
        clean = v.nan_to_num(0, 0, 0)
        o[:, rows] = torch.matmul(w, clean)
        lse[:, rows] = torch.logsumexp(t[:, rows], -1)
        u = torch.finfo(dt_).eps / 2
        reach = torch.matmul(q.abs(), k.nan_to_num(0, 0, 0).abs().transpose(1, 2)).masked_fill(~see, 0)
        dt = ((d + 4) * 2.0 ** -24 * scale * reach.amax(-1))[:, rows, None]
        a = torch.matmul(w, clean.abs())
        under = 2.0 ** -25 * torch.matmul(see.double()[rows], clean.abs()) if dt_ == FP16 else 0.0
        tol[:, rows] = (u + 2 * dt + 2.0 ** -20 + m * 2.0 ** -24) * a + u * o[:, rows].abs() + under \
            + torch.finfo(dt_).tiny * u
    lse_tol = torch.zeros_like(lse)
    if m and rows.any():
        lse_tol[:, rows] = 2 * dt[..., 0] + 2.0 ** -20 + m * 2.0 ** -24 + lse[:, rows].abs() * 2.0 ** -22
    return o.transpose(0, 1), lse.transpose(0, 1), tol.transpose(0, 1), lse_tol.transpose(0, 1)


def make(lens_q, lens_k, hq, hk, d, dtype, seed, fused):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV).to(dtype)

    tq, tk = sum(lens_q), sum(lens_k)
    if fused and lens_q == lens_k:  # the parts of one projection
        qkv = normal(tq, hq + 2 * hk, d)
        return qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    if fused:  # heads outermost
        return normal(hq, tq, d).transpose(0, 1), normal(hk, tk, d).transpose(0, 1), normal(hk, tk, d).transpose(0, 1)
    return normal(tq, hq, d), normal(tk, hk, d), normal(tk, hk, d)


def starts(lens):
    return torch.tensor([0] + list(lens), device=DEV).cumsum(0).to(torch.int32)


def check(o, lse, q, k, v, lens_q, lens_k, causal, scale):
    assert not torch.isnan(o).any()
    q0 = k0 = 0
    for b, (n, m) in enumerate(zip(lens_q, lens_k)):
        eo, el, tol, ltol = exact(q[q0:q0 + n], k[k0:k0 + m], v[k0:k0 + m], causal, scale)
        err = (o[q0:q0 + n].double() - eo).abs()
        assert (err <= tol).all(), (b, n, m, float((err - tol).max()), (err > tol).nonzero()[:3].tolist())
        gl = lse[q0:q0 + n].double()
        empty = torch.isinf(el)
        assert torch.equal(gl[empty], el[empty])
        assert ((gl - el).abs()[~empty] <= ltol[~empty]).all(), (b, n, m)
        q0, k0 = q0 + n, k0 + m


PROMPTS = [
    ([1], 1, 1, 64, BF16), ([1, 2, 3], 8, 8, 128, FP16), ([63, 64, 65], 8, 2, 64, BF16),
    ([127, 128, 129], 5, 1, 128, BF16), ([255, 256, 257, 0, 1], 10, 2, 128, BF16), ([0, 0, 300], 4, 4, 40, BF16),
    ([513, 130], 12, 4, 96, FP16), ([1000], 40, 8, 128, BF16), ([640, 77], 6, 6, 8, BF16), ([700], 20, 1, 128, FP16),
    ([1537], 2, 1, 120, BF16),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,hq,hk,d,dtype", PROMPTS)
def test_prompts(w8a8, lens, hq, hk, d, dtype, causal):
    q, k, v = make(lens, lens, hq, hk, d, dtype, 1 + d + hq, fused=True)
    cu = starts(lens)
    o, lse = w8a8.attention(q, k, v, cu_q=cu, cu_k=cu, causal=causal, lse=True)
    check(o, lse, q, k, v, lens, lens, causal, d ** -0.5)
    assert w8a8.get_device_error() == (0, 0)


MIXED = [
    # (queries, keys): chunks of prompts over what is cached, rows that see nothing, nothing at all
    ([5, 1, 64, 200], [300, 1, 64, 1000], 8, 2, 128, BF16),
    ([300, 4, 129], [20, 0, 128], 4, 2, 128, BF16),
    ([7, 0, 3], [0, 50, 3], 16, 2, 64, FP16),
    ([260, 1, 1], [4100, 9, 700], 5, 1, 128, BF16),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens_q,lens_k,hq,hk,d,dtype", MIXED)
def test_queries_and_keys_of_different_lengths(w8a8, lens_q, lens_k, hq, hk, d, dtype, causal):
    q, k, v = make(lens_q, lens_k, hq, hk, d, dtype, 7 + hq, fused=True)
    o, lse = w8a8.attention(q, k, v, cu_q=starts(lens_q), cu_k=starts(lens_k), causal=causal, scale=0.2, lse=True)
    check(o, lse, q, k, v, lens_q, lens_k, causal, 0.2)


DECODE = [
    ([1], 1, 8, 8, 128, BF16), ([5, 63, 64, 65], 1, 32, 8, 128, BF16), ([300, 0, 129, 2], 1, 5, 1, 64, FP16),
    ([40000], 1, 8, 1, 128, BF16), ([9000, 17, 5000], 2, 40, 8, 128, BF16), ([100, 257, 1], 4, 6, 2, 96, FP16),
    ([4096] * 9, 1, 12, 1, 128, BF16), ([777] * 40, 3, 28, 4, 128, FP16), ([20000, 3], 16, 4, 4, 128, BF16),
    ([512, 100], 30, 20, 4, 64, BF16),
]


@pytest.mark.parametrize("lens,queries,hq,hk,d,dtype", DECODE)
def test_few_queries_over_a_cache(w8a8, lens, queries, hq, hk, d, dtype):
    """A cache with room for more: what lies past each length is NaN."""
    n, cap = len(lens), max(lens) + 37
    q, _, _ = make([queries * n], [1], hq, hk, d, dtype, 3 + hq, fused=False)
    full = make([1], [n * cap], hq, hk, d, dtype, 4 + hq, fused=False)[1:]
    ks, vs = [], []
    for b, m in enumerate(lens):
        for x, parts in zip(full, (ks, vs)):
            parts.append(x[b * cap:b * cap + m].clone())
            x[b * cap + m:(b + 1) * cap] = math.nan
    k_lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
    o, lse = w8a8.attention(q, full[0], full[1], k_lens=k_lens, batch=n, lse=True)
    check(o, lse, q, torch.cat(ks), torch.cat(vs), [queries] * n, lens, True, d ** -0.5)
    # the same call again, and without the statistics: the same bits
    assert torch.equal(o, w8a8.attention(q, full[0], full[1], k_lens=k_lens, batch=n))
    assert w8a8.get_device_error() == (0, 0)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("n,m,hq,hk", [(4, 4, 8, 8), (300, 300, 4, 2), (3, 700, 8, 2), (130, 1000, 2, 1)])
def test_values_that_a_row_does_not_see(w8a8, n, m, hq, hk, bad):
    """A non-finite K or V of the keys from some place on leaves every query
    before it exact."""
    d = 128
    q, k, v = make([n], [m], hq, hk, d, BF16, 11, fused=False)
    at = m - n // 2  # seen by the last n // 2 queries only
    k2, v2 = k.clone(), v.clone()
    k2[at:, :, 3] = bad
    v2[at:, :, 5:9] = bad
    cu_q, cu_k = starts([n]), starts([m])
    o = w8a8.attention(q, k2, v2, cu_q=cu_q, cu_k=cu_k)
    before = n - n // 2
    eo, _, tol, _ = exact(q[:before], k[:m - n + before], v[:m - n + before], True, d ** -0.5)
    assert ((o[:before].double() - eo).abs() <= tol).all()
    # the queries that see a non-finite value show it
    o = w8a8.attention(q, k, v2, cu_q=cu_q, cu_k=cu_k)
    assert not torch.isfinite(o[before:, :, 5:9]).any()
    assert torch.isfinite(o[:, :, 9:]).all() and torch.isfinite(o[:, :, :5]).all()


def test_large_scores_and_equal_keys(w8a8):
    """Scores of +-1000s (the running maximum moves by hundreds), and keys that
    are all alike (uniform weights)."""
    q, k, v = make([300], [300], 4, 2, 64, BF16, 21, fused=False)
    cu = starts([300])
    for scale in (8.0, 1e-3):
        o, lse = w8a8.attention(q, k, v, cu_q=cu, cu_k=cu, scale=scale, lse=True)
        check(o, lse, q, k, v, [300], [300], True, scale)
    k = k[:1].expand(300, 2, 64)
    o, lse = w8a8.attention(q, k, v, cu_q=cu, cu_k=cu, lse=True)
    check(o, lse, q, k, v, [300], [300], True, 0.125)


def test_bounds_in_device_memory_are_clamped(w8a8):
    """Offsets and lengths outside the tensors are taken as their rows' ends."""
    q, k, v = make([40], [50], 4, 2, 64, BF16, 31, fused=False)
    cu_q = torch.tensor([0, 40, 99], dtype=torch.int32, device=DEV)
    cu_k = torch.tensor([-5, 50, 1 << 30], dtype=torch.int32, device=DEV)
    lens = torch.tensor([1 << 30, -3], dtype=torch.int32, device=DEV)
    o, lse = w8a8.attention(q, k, v, cu_q=cu_q, cu_k=cu_k, k_lens=lens, causal=False, lse=True)
    check(o, lse, q, k, v, [40], [50], False, 0.125)


def test_rows_of_no_sequence_are_left_alone(w8a8):
    q, k, v = make([40], [40], 4, 2, 64, BF16, 32, fused=False)
    out = torch.full_like(q, 7.0)
    cu = torch.tensor([8, 20], dtype=torch.int32, device=DEV)
    w8a8.attention(q, k, v, cu_q=cu, cu_k=cu, out=out)
    assert (out[:8] == 7).all() and (out[20:] == 7).all()
    eo, _, tol, _ = exact(q[8:20], k[8:20], v[8:20], True, 0.125)
    assert ((out[8:20].double() - eo).abs() <= tol).all()


def test_strided_output_stream_and_graph(w8a8):
    """Out into a part of a wider tensor, on a side stream, and captured into
    a graph that is replayed on new inputs."""
    q, k, v = make([200, 90], [200, 90], 8, 2, 128, BF16, 41, fused=True)
    cu = starts([200, 90])
    want = w8a8.attention(q, k, v, cu_q=cu, cu_k=cu)
    wide = torch.zeros(290, 12, 128, dtype=BF16, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        w8a8.attention(q, k, v, cu_q=cu, cu_k=cu, out=wide[:, 2:10])
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(wide[:, 2:10], want) and (wide[:, :2] == 0).all() and (wide[:, 10:] == 0).all()
    lens = torch.tensor([20000, 1], dtype=torch.int32, device=DEV)
    kc, vc = make([1], [40000], 8, 2, 128, BF16, 42, fused=False)[1:]
    q1 = make([2], [1], 8, 2, 128, BF16, 43, fused=False)[0]
    graph = torch.cuda.CUDAGraph()
    w8a8.attention(q1, kc, vc, k_lens=lens, batch=2)
    with torch.cuda.graph(graph):
        got = w8a8.attention(q1, kc, vc, k_lens=lens, batch=2)
        prompt = w8a8.attention(q, k, v, cu_q=cu, cu_k=cu)
    for m in (20000, 333, 7777):
        lens[0] = m
        graph.replay()
        assert torch.equal(got, w8a8.attention(q1, kc, vc, k_lens=lens, batch=2))
        assert torch.equal(prompt, want)


@pytest.mark.parametrize("queries", [1, 200])
def test_cache_past_32_bit_offsets(w8a8, queries):
    """The second sequence's keys start past element 2^32 of the cache."""
    hk, d, cap = 8, 128, 4200000
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    k = torch.zeros(2 * cap, hk, d, dtype=BF16, device=DEV)
    v = torch.zeros(2 * cap, hk, d, dtype=BF16, device=DEV)
    m = 900
    q, kk, vv = make([2 * queries], [m], 8, 8, d, BF16, 51, fused=False)
    k[cap:cap + m], v[cap:cap + m] = kk, vv
    assert cap * hk * d > 1 << 32
    lens = torch.tensor([1, m], dtype=torch.int32, device=DEV)
    o = w8a8.attention(q, k, v, k_lens=lens, batch=2)
    eo, _, tol, _ = exact(q[queries:], kk, vv, True, d ** -0.5)
    assert ((o[queries:].double() - eo).abs() <= tol).all()


def test_python_refusals(w8a8):
    q, k, v = make([8], [8], 4, 2, 64, BF16, 61, fused=False)
    cu = starts([8])
    with pytest.raises(TypeError):
        w8a8.attention(q.float(), k.float(), v.float())
    with pytest.raises(TypeError):
        w8a8.attention(q, k.half(), v)
    with pytest.raises(ValueError):
        w8a8.attention(q, k, v[:, :, :32])
    with pytest.raises(ValueError):
        w8a8.attention(q.cpu(), k, v)
    with pytest.raises(ValueError):
        w8a8.attention(q.transpose(1, 2), k, v)
    with pytest.raises(TypeError):
        w8a8.attention(q, k, v, cu_q=cu.long(), cu_k=cu)
    with pytest.raises(ValueError):
        w8a8.attention(q, k, v, cu_q=cu, cu_k=starts([4, 4]))
    with pytest.raises(ValueError):
        w8a8.attention(q, k, v, out=torch.empty(8, 4, 32, dtype=BF16, device=DEV))
    for kw in (dict(batch=3), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan)):
        with pytest.raises(w8a8.W8A8Error):
            w8a8.attention(q, k, v, **kw)
    with pytest.raises(w8a8.W8A8Error, match="WORKSPACE"):
        w8a8.attention(q, k, v, workspace=torch.zeros(256, dtype=torch.uint8, device=DEV))
    assert w8a8.attention(q[:0], k, v).shape == (0, 4, 64)


SCHEDULES = [
    # (lens, Hq, Hk, D, causal): more items than SMs, leftovers taken apart, more than 32
    # sequences, items of one tile between items of two, sequences without a row between
    ([2048, 1000, 257, 77, 1, 1531], 32, 8, 128, True), ([640] * 5, 16, 8, 64, False), ([1024, 1024], 20, 20, 128, False),
    ([1, 130, 0, 63, 257] * 9, 12, 4, 64, True), ([40] * 70, 8, 2, 128, True), ([3000], 16, 1, 64, False),
    ([129, 128, 127] * 11 + [900], 4, 4, 128, True),
]


@pytest.mark.parametrize("lens,hq,hk,d,causal", SCHEDULES)
def test_many_items(w8a8, lens, hq, hk, d, causal):
    q, k, v = make(lens, lens, hq, hk, d, FP16 if d == 64 else BF16, 71 + hq, fused=True)
    cu = starts(lens)
    for _ in range(2):  # the second call finds the counters as the first left them
        o, lse = w8a8.attention(q, k, v, cu_q=cu, cu_k=cu, causal=causal, lse=True)
        check(o, lse, q, k, v, lens, lens, causal, d ** -0.5)
    assert w8a8.get_device_error() == (0, 0)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,m,queries_of", [(700, 700, "prompt"), (90, 2000, "prompt"), (1, 3000, "few"), (6, 1500, "few")])
def test_scores_that_grow_with_the_key(w8a8, n, m, d, queries_of):
    """Every key tile outweighs all before it (and, for half of the heads, every
    tile is outweighed by the first): the softmax's reference moves each time."""
    q, k, v = make([n], [m], 4, 2, d, BF16, 81 + d, fused=False)
    ramp = torch.linspace(0, 40, m, device=DEV)[:, None]
    k[:, 0, :1] += ramp.to(BF16)
    k[:, 1, :1] -= ramp.to(BF16)
    q[:, :, 0] = 8.0
    cu_q, cu_k = starts([n]), starts([m])
    for causal in (True, False):
        o, lse = w8a8.attention(q, k, v, cu_q=cu_q, cu_k=cu_k, causal=causal, scale=1.0, lse=True)
        check(o, lse, q, k, v, [n], [m], causal, 1.0)
    assert w8a8.get_device_error() == (0, 0)


def test_broadcast_keys_and_many_heads_a_group(w8a8):
    """KV heads that are one head expanded, and more query heads on a KV head
    than a tile of rows holds."""
    q, k, v = make([150], [200], 6, 1, 64, BF16, 91, fused=False)
    cu_q, cu_k = starts([150]), starts([200])
    o, lse = w8a8.attention(q, k.expand(200, 3, 64), v.expand(200, 3, 64), cu_q=cu_q, cu_k=cu_k, lse=True)
    check(o, lse, q, k, v, [150], [200], True, 0.125)
    q, k, v = make([3], [900], 300, 2, 64, FP16, 92, fused=False)
    o, lse = w8a8.attention(q, k, v, cu_q=starts([3]), cu_k=starts([900]), lse=True)
    check(o, lse, q, k, v, [3], [900], True, 0.125)


def test_calls_on_streams_of_their_own(w8a8):
    """Overlapping calls on several streams, each with its stream's workspace."""
    jobs = []
    for i in range(4):
        lens = torch.tensor([20000 + 777 * i, 100], dtype=torch.int32, device=DEV)
        q = make([2], [1], 8, 2, 128, BF16, 101 + i, fused=False)[0]
        kc, vc = make([1], [50000], 8, 2, 128, BF16, 105 + i, fused=False)[1:]
        jobs.append((q, kc, vc, lens, w8a8.attention(q, kc, vc, k_lens=lens, batch=2)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(10):
        got = []
        for s, (q, kc, vc, lens, _) in zip(streams, jobs):
            with torch.cuda.stream(s):
                got.append(w8a8.attention(q, kc, vc, k_lens=lens, batch=2))
        torch.cuda.synchronize()
        assert all(torch.equal(a, job[4]) for a, job in zip(got, jobs))


@pytest.mark.parametrize("hq,hk,d,dtype", [(32, 8, 128, BF16), (8, 2, 64, FP16), (6, 6, 72, BF16)])
def test_caches_with_many_items(w8a8, hq, hk, d, dtype):
    """More sequences than CTAs work on at once, of 0 to 700 keys; twice, as the
    second call finds the counters as the first left them."""
    lens = [(37 * i * i + 11 * i) % 701 for i in range(260)]
    lens[5] = 0
    cap = 704
    q = make([1] * 260, [1], hq, hk, d, dtype, 111, fused=False)[0]
    k, v = make([1], [260 * cap], hq, hk, d, dtype, 112, fused=False)[1:]
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    for _ in range(2):
        o, lse = w8a8.attention(q, k, v, k_lens=n, batch=260, lse=True)
        for b in list(range(0, 260, 13)) + [5, 259]:
            rows = slice(b * cap, b * cap + lens[b])
            check(o[b:b + 1], lse[b:b + 1], q[b:b + 1], k[rows], v[rows], [1], [lens[b]], True, d ** -0.5)
    assert w8a8.get_device_error() == (0, 0)


@pytest.mark.parametrize("lens,queries,hq,hk,d", [
    ([300] * 8, 1, 32, 8, 128), ([420, 367, 0, 172], 1, 32, 8, 64), ([4871], 4, 12, 1, 128), ([64, 65, 1, 640, 0, 129], 2, 28, 4, 72),
    ([3471, 2395, 2544, 2414], 1, 12, 1, 64), ([500] * 31 + [7000], 1, 16, 2, 128), ([130] * 32, 3, 8, 8, 128), ([90000, 3, 70], 1, 8, 8, 128),
])
def test_caches_cut_into_pieces(w8a8, lens, queries, hq, hk, d):
    """Few tiles of keys for many CTAs: whole ranges an item, and the joins; twice,
    as the second call finds the counters as the first left them."""
    n, cap = len(lens), max(lens) + 5
    q = make([queries] * n, [1], hq, hk, d, BF16, 121, fused=False)[0]
    k, v = make([1], [n * cap], hq, hk, d, BF16, 122, fused=False)[1:]
    on_gpu = torch.tensor(lens, dtype=torch.int32, device=DEV)
    for _ in range(2):
        o, lse = w8a8.attention(q, k, v, k_lens=on_gpu, batch=n, lse=True)
        for b in range(n):
            rows, mine = slice(b * cap, b * cap + lens[b]), slice(b * queries, (b + 1) * queries)
            check(o[mine], lse[mine], q[mine], k[rows], v[rows], [queries], [lens[b]], True, d ** -0.5)
    assert w8a8.get_device_error() == (0, 0)
