"""Copies of pages and forks of sequences: exact."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, FP16 = torch.bfloat16, torch.float16


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def make(n, pages, shape, dtype, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return [torch.randn(pages, *shape, generator=g, device=DEV).to(dtype) for _ in range(n)]


@pytest.mark.parametrize("n,pages,shape,dtype,moves", [
    (1, 2, (8, 1, 8), BF16, 1), (2, 9, (16, 2, 64), FP16, 4), (7, 40, (64, 8, 128), BF16, 19), (3, 11, (24, 3, 40), BF16, 5),
    (200, 30, (16, 1, 64), BF16, 11), (400, 4, (8, 1, 16), FP16, 2), (2, 5, (5000, 2, 128), BF16, 2),
    (4, 12, (16, 8), torch.uint8, 6), (2, 300, (16, 2, 64), torch.float32, 150)])
def test_copy(w8a8, n, pages, shape, dtype, moves):
    caches = make(n, pages, shape, dtype, n + pages)
    order = torch.randperm(pages, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)).to(torch.int32)
    src, dst = order[:moves].contiguous(), order[moves:2 * moves].contiguous()
    want = [c.clone() for c in caches]
    for c in want:
        c[dst.long()] = c[src.long()]
    w8a8.copy_pages(caches, src, dst)
    for c, x in zip(caches, want):
        assert torch.equal(c, x)


def test_copy_within_wider_tensors(w8a8):
    """K and V of a page side by side, pages of heads first, and a tuple of all of them."""
    both = make(1, 20, (2, 16, 4, 64), BF16, 3)[0]
    heads = make(1, 20, (4, 16, 64), BF16, 4)[0].transpose(1, 2)
    keep, keep_heads = both.clone(), heads.clone()
    src, dst = ints(3, 19, 3), ints(0, 7, 9)
    w8a8.copy_pages((both[:, 0], heads), src, dst)
    keep[:, 0][dst.long()] = keep[:, 0][src.long()]
    keep_heads[dst.long()] = keep_heads[src.long()]
    assert torch.equal(both, keep) and torch.equal(heads, keep_heads)


def test_copy_of_nothing(w8a8):
    caches = make(2, 6, (16, 2, 64), BF16, 5)
    want = [c.clone() for c in caches]
    w8a8.copy_pages(caches, ints(-1, 6, 2, 1 << 30, 4, 3), ints(0, 1, -1, 2, 6, 3))
    w8a8.copy_pages(caches, ints(), ints())
    w8a8.copy_pages([c[:0] for c in caches], ints(0), ints(1))
    for c, x in zip(caches, want):
        assert torch.equal(c, x)


def test_copy_past_32_bits(w8a8):
    pages = (5 << 30) // (64 * 8 * 128 * 2) + 1
    c = torch.zeros(pages, 64, 8, 128, dtype=BF16, device=DEV)
    x = torch.randn(2, 64, 8, 128, device=DEV).to(BF16)
    c[2], c[pages - 1] = x[0], x[1]
    w8a8.copy_pages([c], ints(2, pages - 1), ints(pages - 2, 5))
    assert torch.equal(c[pages - 2], x[0]) and torch.equal(c[5], x[1])


def forked(caches, table, lens, src, dst, new, page):
    """The definition, pair by pair on the host."""
    pages, columns, rows = caches[0].shape[0], table.shape[1], table.shape[0]
    table, lens = table.clone(), lens.clone()
    caches = [c.clone() for c in caches]
    for a, b, p in zip(src.tolist(), dst.tolist(), new.tolist()):
        if a == b or not (0 <= a < rows and 0 <= b < rows and 0 <= p < pages):
            continue
        n = min(max(int(lens[a]), 0), columns * page)
        full = n // page
        if n % page:
            old = int(table[a, full])
            if 0 <= old < pages:
                for c in caches:
                    c[p] = c[old]
        table[b, :full] = table[a, :full]
        if full < columns:
            table[b, full] = p
        lens[b] = n
    return caches, table, lens


@pytest.mark.parametrize("n,page,shape,columns", [(1, 8, (8, 1, 8), 1), (6, 16, (16, 2, 64), 5), (300, 64, (64, 1, 32), 9),
                                                  (2, 40, (40, 8, 128), 700)])
def test_fork(w8a8, n, page, shape, columns):
    g = torch.Generator(device=DEV).manual_seed(n)
    rows, pages = 14, 60
    caches = make(n, pages, shape, BF16, 7)
    # part of a wider table, columns behind it are nobody's
    wide = torch.randint(0, pages - 20, (rows, columns + 3), generator=g, device=DEV).to(torch.int32)
    table = wide[:, :columns]
    full = columns * page
    lens = ints(0, 1, page - 1, page, page + 1, full - 1, full, full + 1, -3, 1 << 30, 5, 6, 7, 8)
    table[4, 0] = -1 if columns == 1 else table[4, 0]
    src = ints(0, 1, 2, 3, 4, 5, 6, 6, -1, 20, 4)
    dst = ints(10, 11, 12, 13, 8, 9, 7, 14, 3, 2, 4)
    new = torch.arange(pages - len(src), pages, dtype=torch.int32, device=DEV)
    keep = wide.clone()
    want = forked(caches, table, lens, src, dst, new, page)
    w8a8.fork_sequences(caches, table, lens, src, dst, new, page)
    assert torch.equal(table, want[1]) and torch.equal(lens, want[2])
    assert torch.equal(wide[:, columns:], keep[:, columns:])
    for c, x in zip(caches, want[0]):
        assert torch.equal(c, x)


def test_one_source_of_many_and_pages_that_are_not_there(w8a8):
    caches = make(4, 30, (16, 2, 64), FP16, 9)
    table = torch.full((8, 4), -1, dtype=torch.int32, device=DEV)
    table[0, :3] = ints(4, 2, 9)
    lens = ints(37, 0, 0, 0, 0, 0, 0, 0)
    src, dst, new = ints(0, 0, 0, 0), ints(1, 2, 3, 4), ints(20, 21, -1, 30)
    want = forked(caches, table, lens, src, dst, new, 16)
    w8a8.fork_sequences(caches, table, lens, src, dst, new, 16)
    assert torch.equal(table, want[1]) and torch.equal(lens, want[2])
    assert lens.tolist() == [37, 37, 37, 0, 0, 0, 0, 0]
    for c, x in zip(caches, want[0]):
        assert torch.equal(c, x)


def test_captured(w8a8):
    caches = make(3, 20, (16, 2, 64), BF16, 11)
    src, dst = ints(1, 2), ints(10, 11)
    w8a8.copy_pages([c.clone() for c in caches], src, dst)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w8a8.copy_pages(caches, src, dst)
    for a, b in ((3, 12), (5, 13), (-1, 14)):
        src.copy_(ints(a, a))
        dst.copy_(ints(b, b + 3))
        want = [c.clone() for c in caches]
        if a >= 0:
            for c in want:
                c[b] = c[b + 3] = c[a]
        graph.replay()
        for c, x in zip(caches, want):
            assert torch.equal(c, x)
