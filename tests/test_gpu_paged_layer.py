"""Int8TransformerLayer over pages: the operators together, as a server uses them."""
import pytest
import torch

from test_gpu_attention import check, exact, starts

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16
WIDTH, HIDDEN, HEADS, KV_HEADS, DIM, PAGE, PAGES = 512, 1024, 8, 2, 64, 16, 60


def make(w8a8, norms):
    g = torch.Generator(device=DEV).manual_seed(3)

    def w(*shape, std=0.04):
        return (torch.randn(shape, generator=g, device=DEV) * std).to(BF16)

    more = dict(q_norm=1 + w(DIM, std=0.2), k_norm=1 + w(KV_HEADS, DIM, std=0.2)) if norms else {}
    return w8a8.Int8TransformerLayer(
        w((HEADS + 2 * KV_HEADS) * DIM, WIDTH), w(WIDTH, HEADS * DIM), w(HIDDEN, WIDTH), w(WIDTH, HIDDEN), HEADS,
        KV_HEADS, 1 + w(WIDTH, std=0.1), 1 + w(WIDTH, std=0.1), w8a8.rotary_frequencies(DIM), **more)


class Server:
    """Sequences in pages: what a caller keeps (free pages, tables, lengths)."""

    def __init__(self, layer, rows, columns, seed):
        self.layer = layer
        self.k, self.v = layer.new_pages(PAGES, PAGE)
        g = torch.Generator().manual_seed(seed)
        self.free = torch.randperm(PAGES, generator=g).tolist()
        self.table = torch.full((rows, columns), -1, dtype=torch.int32, device=DEV)
        self.lens = torch.zeros(rows, dtype=torch.int32, device=DEV)

    def step(self, tokens, **kw):
        """tokens: one [n, WIDTH] for each row."""
        pos, slots = [], []
        for b, x in enumerate(tokens):
            n, m = x.shape[0], int(self.lens[b])
            at = torch.arange(m, m + n)
            for column in range(-(-m // PAGE), -(-(m + n) // PAGE)):
                if int(self.table[b, column]) < 0:
                    self.table[b, column] = self.free.pop()
            pos.append(at)
            slots.append(self.table[b].cpu().long()[at // PAGE] * PAGE + at % PAGE)
            self.lens[b] += n
        x = torch.cat(tokens)
        args = (x, torch.cat(pos).to(DEV), self.k, self.v, torch.cat(slots).to(DEV), self.lens, len(tokens))
        kw = dict(cu_q=starts([t.shape[0] for t in tokens]), page_table=self.table, **kw)
        return self.layer(*args, **kw), args, kw

    def rows_of(self, b):
        m = int(self.lens[b])
        i = torch.arange(m, device=DEV)
        at = self.table[b].long()[i // PAGE], i % PAGE
        return self.k[at], self.v[at]


@pytest.mark.parametrize("norms", [True, False])
def test_is_its_operators_in_turn(w8a8, norms):
    """A prompt's chunk, a whole prompt and a single token in one call: bit for bit the
    public calls one after another, and the attention within its tolerance."""
    layer = make(w8a8, norms)
    s = Server(layer, 3, 20, 1)
    g = torch.Generator(device=DEV).manual_seed(2)
    token = lambda n: torch.randn(n, WIDTH, generator=g, device=DEV).to(BF16)
    s.step([token(100), token(0), token(37)])
    before = s.k.clone(), s.v.clone()
    y, args, kw = s.step([token(70), token(90), token(1)])
    x, pos, _, _, slots, lens, _ = args
    qkv = layer.qkv(x).view(-1, HEADS + 2 * KV_HEADS, DIM)
    q, k, v = qkv.split((HEADS, KV_HEADS, KV_HEADS), dim=1)
    if norms:
        q = w8a8.qk_norm_rotary_append(q, k, v, pos, layer.frequencies, *before, slots, layer.q_norm, layer.k_norm)
    else:
        rows = (-1, KV_HEADS, DIM)
        q = w8a8.rotary_append(q, k, v, pos, layer.frequencies, before[0].view(rows), before[1].view(rows), slots)
    assert torch.equal(before[0], s.k) and torch.equal(before[1], s.v)
    a, lse = w8a8.paged_attention(q, s.k, s.v, s.table, lens, cu_q=kw["cu_q"], lse=True)
    ks, vs = zip(*(s.rows_of(b) for b in range(3)))
    check(a, lse, q, torch.cat(ks), torch.cat(vs), [70, 90, 1], [170, 90, 38], True, DIM ** -0.5)
    h, _, _, _, u = w8a8.residual_norm_quant(x, layer.out(a.view(-1, HEADS * DIM)), gamma=layer.ffn_norm, image=False,
                                             y=True)
    assert torch.equal(y, h + layer.ffn(u))
    assert torch.isfinite(y).all() and w8a8.get_device_error() == (0, 0)


@pytest.mark.parametrize("norms", [True, False])
def test_pages_hold_what_a_dense_cache_holds(w8a8, norms):
    """The same tokens into a dense cache, in other steps: the same keys and values."""
    layer = make(w8a8, norms)
    s = Server(layer, 2, 10, 4)
    x = [torch.randn(n, WIDTH, device=DEV).to(BF16) for n in (83, 21)]
    s.step([x[0][:40], x[1][:20]])
    s.step([x[0][40:82], x[1][20:20]])
    s.step([x[0][82:], x[1][20:]])
    cap = 100
    kc, vc = layer.new_cache(2, cap)
    pos = torch.cat([torch.arange(83), torch.arange(21)]).to(DEV)
    slots = pos + cap * (torch.arange(104, device=DEV) >= 83)
    layer(torch.cat(x), pos, kc, vc, slots, s.lens, 2, cu_q=starts([83, 21]))
    for b, n in enumerate((83, 21)):
        k, v = s.rows_of(b)
        assert torch.equal(k, kc[b * cap:b * cap + n]) and torch.equal(v, vc[b * cap:b * cap + n])


def test_fork_go_on_and_compact(w8a8):
    """A prompt, two more sequences forked from it, each going on with tokens of its
    own (the decoding step captured into a graph), then the pages compacted: what
    every step computes stays what the formula says over each sequence's own tokens."""
    layer = make(w8a8, True)
    s = Server(layer, 3, 8, 6)
    g = torch.Generator(device=DEV).manual_seed(7)
    token = lambda n: torch.randn(n, WIDTH, generator=g, device=DEV).to(BF16)
    prompt = token(53)
    s.step([prompt, token(0), token(0)])
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)
    new = [s.free.pop(), s.free.pop()]
    w8a8.fork_sequences([s.k, s.v], s.table, s.lens, ints([0, 0]), ints([1, 2]), ints(new), page_size=PAGE)
    assert s.lens.tolist() == [53, 53, 53]
    for b in (1, 2):
        assert s.table[b, :3].tolist() == s.table[0, :3].tolist() and int(s.table[b, 3]) == new[b - 1]
        assert all(torch.equal(a, c) for a, c in zip(s.rows_of(b), s.rows_of(0)))
    own = [[prompt] for _ in range(3)]

    def checked(y, args, kw, queries):
        x, pos, *_ = args
        q = layer.qkv(x).view(-1, HEADS + 2 * KV_HEADS, DIM)[:, :HEADS]
        q, _ = w8a8.qk_norm_rotary(q, None, pos, layer.frequencies, q_gamma=layer.q_norm)
        a = w8a8.paged_attention(q, s.k, s.v, s.table, s.lens, cu_q=kw["cu_q"])
        at = 0
        for b, n in enumerate(queries):
            # keys and values of this sequence's tokens, from nothing
            t = torch.cat(own[b])
            _, k, v = layer.qkv(t).view(-1, HEADS + 2 * KV_HEADS, DIM).split((HEADS, KV_HEADS, KV_HEADS), dim=1)
            k, _ = w8a8.qk_norm_rotary(k, None, torch.arange(t.shape[0], device=DEV), layer.frequencies,
                                       q_gamma=layer.k_norm)
            assert torch.equal(s.rows_of(b)[0], k) and torch.equal(s.rows_of(b)[1], v)
            o, _, tol, _ = exact(q[at:at + n], k, v, True, DIM ** -0.5)
            assert ((a[at:at + n].double() - o).abs() <= tol).all()
            at += n

    for n in ((1, 1, 1), (3, 1, 20), (1, 1, 1)):
        more = [token(i) for i in n]
        for b in range(3):
            own[b].append(more[b])
        checked(*s.step(more), n)
    # the used pages to the front
    used = sorted({int(v) for b in range(3) for v in s.table[b, :-(-int(s.lens[b]) // PAGE)]})
    holes = [i for i in range(len(used)) if i not in used]
    moved = [i for i in used if i >= len(used)]
    src, dst = ints(moved), ints(holes)
    w8a8.copy_pages([s.k, s.v], src, dst)
    to = torch.arange(PAGES, dtype=torch.int32, device=DEV)
    to[src.long()] = dst
    s.table[:] = torch.where(s.table >= 0, to[s.table.clamp(min=0).long()], s.table)
    s.free = list(range(len(used), PAGES))
    for cache in (s.k, s.v):
        cache[len(used):] = float("nan")  # nobody's any more
    more = [token(1) for _ in range(3)]
    for b in range(3):
        own[b].append(more[b])
    y, args, kw = s.step(more, max_queries=1)
    checked(y, args, kw, (1, 1, 1))
    # the same step captured, and replayed twice
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(*args, **kw)
    for _ in range(2):
        out.zero_()
        graph.replay()
        assert torch.equal(out, y)
    assert w8a8.get_device_error() == (0, 0)


def test_refusals(w8a8):
    layer = make(w8a8, True)
    k, v = layer.new_pages(4, PAGE)
    x = torch.zeros(2, WIDTH, dtype=BF16, device=DEV)
    z = torch.zeros(2, dtype=torch.int64, device=DEV)
    with pytest.raises(ValueError, match="page_table"):
        layer(x, z, k, v, z, z.int(), 2, page_table=torch.zeros(3, 1, dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError, match="q_norm and k_norm"):
        w = torch.zeros(12 * DIM, WIDTH, dtype=BF16, device=DEV)
        w8a8.Int8TransformerLayer(w, w, w, w, HEADS, KV_HEADS, w[0], w[0], layer.frequencies, q_norm=w[0, :DIM])
