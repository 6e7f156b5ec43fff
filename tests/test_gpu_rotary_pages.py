"""Rotary positions with K and V written to caches in pages, of any strides: bit for bit what
the same tokens get in a cache of rows; and a layer over such pages."""
import pytest
import torch

from test_gpu_attention import starts
from test_gpu_paged_layer import HEADS, KV_HEADS, DIM, PAGE, PAGES, WIDTH, make

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, FP16 = torch.bfloat16, torch.float16


def pages_of(layout, pages, page, hk, d, dtype):
    """Caches in pages full of nines, and the tensors that they are views of."""
    if layout == "token":
        whole = [torch.full((pages, page, hk, d), 9.0, dtype=dtype, device=DEV) for _ in range(2)]
        return whole, whole
    if layout == "head":  # every head's rows of a page together
        whole = [torch.full((pages, hk, page, d), 9.0, dtype=dtype, device=DEV) for _ in range(2)]
        return [t.transpose(1, 2) for t in whole], whole
    if layout == "row":  # the same row of all pages together
        whole = [torch.full((page, pages, hk, d), 9.0, dtype=dtype, device=DEV) for _ in range(2)]
        return [t.transpose(0, 1) for t in whole], whole
    # K and V of a page side by side, in a wider row
    both = torch.full((pages, 2, page, hk, d + 8), 9.0, dtype=dtype, device=DEV)
    return [both[:, 0, :, :, :d], both[:, 1, :, :, :d]], [both]


LAYOUTS = ["token", "head", "row", "pair"]


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("t,pages,page,hq,hk,d,rot,dtype,turn", [
    (1, 1, 1, 4, 1, 16, 16, BF16, "half"), (37, 9, 16, 8, 2, 128, 128, BF16, "half"),
    (60, 5, 24, 5, 5, 72, 32, FP16, "interleaved"), (1900, 300, 8, 32, 8, 64, 64, BF16, "half"),
    (3, 1, 1000, 2, 1, 256, 96, FP16, "half")])
def test_pages_hold_what_rows_hold(w8a8, t, pages, page, hq, hk, d, rot, dtype, turn, layout):
    g = torch.Generator(device=DEV).manual_seed(t + d)
    qkv = torch.randn(t, hq + 2 * hk, d, generator=g, device=DEV).to(dtype)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    pos = torch.randint(0, 1 << 20, (t,), generator=g, device=DEV)
    freqs = w8a8.rotary_frequencies(rot)
    rows = pages * page
    slots = torch.randperm(rows + t, generator=g, device=DEV)[:t]  # some behind the cache
    slots[::7] = torch.where(torch.arange(len(slots[::7]), device=DEV) % 2 == 0, slots[::7], -1)
    want = [torch.full((rows, hk, d), 9.0, dtype=dtype, device=DEV) for _ in range(2)]
    q1 = w8a8.rotary_append(q, k, v, pos, freqs, *want, slots, layout=turn, amplitude=1.25)
    caches, whole = pages_of(layout, pages, page, hk, d, dtype)
    q2 = w8a8.rotary_append(q, k, v, pos, freqs, *caches, slots, layout=turn, amplitude=1.25)
    assert torch.equal(q1, q2)
    for c, x in zip(caches, want):
        assert torch.equal(c.reshape(rows, hk, d), x)
        c.fill_(9.0)
    assert all((x == 9).all() for x in whole)  # nothing else was written


def test_rows_past_32_bits(w8a8):
    page, hk, d = 32, 4, 128
    pages = (5 << 30) // (page * hk * d * 2) + 1
    kc, vc = (torch.zeros(pages, page, hk, d, dtype=BF16, device=DEV) for _ in range(2))
    q, k, v = (torch.randn(3, h, d, device=DEV).to(BF16) for h in (8, hk, hk))
    pos = torch.arange(3, device=DEV)
    slots = torch.tensor([pages * page - 1, 5, pages * page // 2 + 3], device=DEV)
    freqs = w8a8.rotary_frequencies(d)
    w8a8.rotary_append(q, k, v, pos, freqs, kc, vc, slots)
    _, k1 = w8a8.rotary(q, k, pos, freqs)
    assert torch.equal(kc.flatten(0, 1)[slots], k1) and torch.equal(vc.flatten(0, 1)[slots], v)


def test_captured(w8a8):
    freqs = w8a8.rotary_frequencies(64)
    q, k, v = (torch.randn(5, h, 64, device=DEV).to(BF16) for h in (4, 2, 2))
    pos, slots = torch.arange(5, device=DEV), torch.tensor([9, 3, -1, 30, 0], device=DEV)
    caches = [torch.zeros(2, 2, 16, 64, dtype=BF16, device=DEV).transpose(1, 2) for _ in range(4)]
    w8a8.rotary_append(q, k, v, pos, freqs, caches[2], caches[3], slots)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = w8a8.rotary_append(q, k, v, pos, freqs, caches[0], caches[1], slots)
    graph.replay()
    for _ in range(3):
        q.normal_()
        k.normal_()
        pos += 1000
        slots.copy_(slots.roll(1))
        graph.replay()
        assert torch.equal(out, w8a8.rotary_append(q, k, v, pos, freqs, caches[2], caches[3], slots))
        assert torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])


def test_refusals(w8a8):
    freqs = w8a8.rotary_frequencies(64)
    q, kv = torch.zeros(3, 4, 64, dtype=BF16, device=DEV), torch.zeros(3, 2, 64, dtype=BF16, device=DEV)
    z = torch.zeros(3, dtype=torch.int64, device=DEV)
    pages = torch.zeros(4, 16, 2, 64, dtype=BF16, device=DEV)
    call = lambda a, b: w8a8.rotary_append(q, kv, kv, z, freqs, a, b, z)
    for a, b in ((pages, pages[:, :8]), (pages, pages.view(64, 2, 64)), (pages[:, :, :1], pages[:, :, :1])):
        with pytest.raises(ValueError, match="both caches"):
            call(a, b)
    with pytest.raises(ValueError, match=r"k_cache must be \[pages, page_size, KV heads, dim\] or \[rows, KV heads"):
        call(pages[0, 0], pages[0, 0])
    with pytest.raises(w8a8.W8A8Error):  # pages on one another
        call(pages[:1].expand(4, -1, -1, -1), pages)
    with pytest.raises(ValueError, match="k_cache requires a gradient"):
        call(pages.clone().requires_grad_(), pages)


@pytest.mark.parametrize("norms", [True, False])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_layer(w8a8, layout, norms):
    """A prompt and a single token, then a token of each: what dense pages give."""
    layer = make(w8a8, norms)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)
    table = ints([[7, 50, 3, 12], [9, 8, 0, 1]])
    results = []
    for caches in (layer.new_pages(PAGES, PAGE), pages_of(layout, PAGES, PAGE, KV_HEADS, DIM, BF16)[0]):
        g = torch.Generator(device=DEV).manual_seed(5)
        out = []
        for at, n in (((0, 0), (50, 1)), ((50, 1), (1, 1))):
            pos = torch.cat([torch.arange(a, a + i, device=DEV) for a, i in zip(at, n)])
            row = torch.repeat_interleave(torch.arange(2, device=DEV), torch.tensor(n, device=DEV))
            slots = table.long()[row, pos // PAGE] * PAGE + pos % PAGE
            x = torch.randn(sum(n), WIDTH, generator=g, device=DEV).to(BF16)
            out.append(layer(x, pos, *caches, slots, ints([a + i for a, i in zip(at, n)]), 2, cu_q=starts(list(n)),
                             page_table=table))
        results.append((*out, caches[0][table[0].long()].reshape(-1, KV_HEADS, DIM)[:51],
                        caches[1][table[0].long()].reshape(-1, KV_HEADS, DIM)[:51]))
    for a, b in zip(*results):
        assert torch.equal(a, b) and torch.isfinite(a).all()
    assert w8a8.get_device_error() == (0, 0)
