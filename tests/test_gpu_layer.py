"""Int8TransformerLayer: the operators together, as a program uses them."""
import pytest
import torch

from test_gpu_attention import exact, starts

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16
WIDTH, HIDDEN, HEADS, KV_HEADS, DIM, CAPACITY = 512, 1024, 8, 2, 64, 300


@pytest.fixture(scope="module")
def layer(w8a8):
    g = torch.Generator(device=DEV).manual_seed(3)

    def w(*shape, std=0.04):
        return (torch.randn(shape, generator=g, device=DEV) * std).to(BF16)

    return w8a8.Int8TransformerLayer(
        w((HEADS + 2 * KV_HEADS) * DIM, WIDTH), w(WIDTH, HEADS * DIM), w(HIDDEN, WIDTH), w(WIDTH, HIDDEN), HEADS,
        KV_HEADS, 1 + w(WIDTH, std=0.1), 1 + w(WIDTH, std=0.1), w8a8.rotary_frequencies(DIM))


def tokens(lens, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(sum(lens), WIDTH, generator=g, device=DEV).to(BF16)
    pos = torch.cat([torch.arange(n, device=DEV) for n in lens])
    seq = torch.cat([torch.full((n,), b, device=DEV) for b, n in enumerate(lens)])
    return x, pos, seq * CAPACITY + pos


def test_is_its_operators_in_turn(w8a8, layer):
    """Bit for bit the public calls one after another, and the attention in
    between within its tolerance of the formula over the cache."""
    lens = [200, 1, 77]
    x, pos, slots = tokens(lens, 1)
    k_lens, cu = torch.tensor(lens, dtype=torch.int32, device=DEV), starts(lens)
    kc, vc = layer.new_cache(3, CAPACITY)
    y = layer(x, pos, kc, vc, slots, k_lens, 3, cu_q=cu)
    qkv = layer.qkv(x).view(-1, HEADS + 2 * KV_HEADS, DIM)
    q, k = w8a8.rotary(qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV_HEADS], pos, layer.frequencies)
    assert torch.equal(kc[slots], k) and torch.equal(vc[slots], qkv[:, HEADS + KV_HEADS:])
    a = w8a8.attention(q, kc, vc, cu_q=cu, k_lens=k_lens)
    at = 0
    for b, n in enumerate(lens):
        rows = slice(b * CAPACITY, b * CAPACITY + n)
        o, _, tol, _ = exact(q[at:at + n], kc[rows], vc[rows], True, DIM ** -0.5)
        assert ((a[at:at + n].double() - o).abs() <= tol).all()
        at += n
    h, _, _, _, u = w8a8.residual_norm_quant(x, layer.out(a.view(-1, HEADS * DIM)), gamma=layer.ffn_norm, image=False,
                                             y=True)
    assert torch.equal(y, h + layer.ffn(u))
    assert torch.isfinite(y).all() and w8a8.get_device_error() == (0, 0)


def test_single_tokens_continue_a_prompt(w8a8, layer):
    """Two sequences: a prompt at once, then token by token (captured into a
    graph and replayed).  The cache is that of the whole run, bit for bit (the
    W8A8 Linear gives the same bits for one token as for many), and each new
    token's attention is within its tolerance of the formula."""
    prompt, more = [40, 9], 5
    lens = [n + more for n in prompt]
    x, pos, slots = tokens(lens, 2)
    whole = layer.new_cache(2, CAPACITY)
    layer(x, pos, *whole, slots, torch.tensor(lens, dtype=torch.int32, device=DEV), 2, cu_q=starts(lens))
    start = [0, lens[0]]
    first = torch.cat([torch.arange(s, s + n, device=DEV) for s, n in zip(start, prompt)])
    cache = layer.new_cache(2, CAPACITY)
    k_lens = torch.tensor(prompt, dtype=torch.int32, device=DEV)
    layer(x[first], pos[first], *cache, slots[first], k_lens, 2, cu_q=starts(prompt))
    # static inputs of one step
    sx, sp, ss = x[:2].clone(), pos[:2].clone(), slots[:2].clone()
    scratch = layer.new_cache(2, CAPACITY)
    for c, s in zip(scratch, cache):
        c.copy_(s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(sx, sp, *scratch, ss, k_lens, 2)  # warm-up, on a copy of the cache
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(sx, sp, *cache, ss, k_lens, 2)
    for step in range(more):
        at = torch.tensor([s + n + step for s, n in zip(start, prompt)], device=DEV)
        sx.copy_(x[at])
        sp.copy_(pos[at])
        ss.copy_(slots[at])
        k_lens += 1
        graph.replay()
        got = out.clone()
        assert torch.equal(got, layer(sx, sp, *cache, ss, k_lens, 2))  # the same token once more
        qkv = layer.qkv(sx).view(2, -1, DIM)
        q, _ = w8a8.rotary(qkv[:, :HEADS], None, sp, layer.frequencies)
        a = w8a8.attention(q, *cache, k_lens=k_lens, batch=2)
        for b in range(2):
            rows = slice(b * CAPACITY, b * CAPACITY + prompt[b] + step + 1)
            o, _, tol, _ = exact(q[b:b + 1], whole[0][rows], whole[1][rows], True, DIM ** -0.5)
            assert ((a[b:b + 1].double() - o).abs() <= tol).all()
    for c, w in zip(cache, whole):
        assert torch.equal(c, w)


def test_refusals(w8a8, layer):
    w = torch.zeros(700, WIDTH, dtype=BF16, device=DEV)
    with pytest.raises(ValueError):
        w8a8.Int8TransformerLayer(w, w, w, w, HEADS, KV_HEADS, w[0], w[0], layer.frequencies)
    with pytest.raises(ValueError):
        w8a8.Int8TransformerLayer(w[:10 * DIM], w, w, w, 4, 3, w[0], w[0], layer.frequencies)
