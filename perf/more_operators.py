"""Measured cases of the operators around a paged cache.

Four operators: `paged_attention` (new tokens, from one to a long chunk of a
prompt for each sequence, over caches in pages), `qk_norm_rotary` /
`qk_norm_rotary_append` (norms of the query and key heads with the rotary
positions, and the cache rows written with them), `copy_pages` (pages moved
within every layer's caches) and `fork_sequences` (a sequence continued more
than once: its page table shared, its last page copied).  `run` computes a case
in plain 32-bit torch operations, or, where `own` is true, with the package's
entry points.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _ragged(n, longest):
    return ",".join(str(1 + (i * 2654435761 + 977) % longest) for i in range(n))


def listed():
    return [
        # -- attention over paged caches
        # the next chunk of a long prompt that is taken in piece by piece
        dict(name="paged_chunk_512", op="attention", queries="512", lens="33280", page=64, heads=40, kv_heads=8,
             dim=128, causal=True, dtype="bf16"),
        # a serving step: two prompts' chunks among requests that each add one token
        dict(name="paged_mixed_26", op="attention", queries="700,333" + 24 * ",1", lens="4796,333," + _ragged(24, 6000),
             page=32, heads=32, kv_heads=8, dim=128, causal=True, dtype="bf16"),
        # draft tokens checked for a batch of requests
        dict(name="paged_draft_16x5", op="attention", queries="5" + 15 * ",5", lens=_ragged(16, 8000), page=16,
             heads=28, kv_heads=4, dim=128, causal=True, dtype="bf16"),
        # a batch in which every request adds one token, small pages
        dict(name="paged_single_48", op="attention", queries="1" + 47 * ",1", lens=_ragged(48, 8192), page=16, heads=32,
             kv_heads=8, dim=128, causal=True, dtype="bf16"),
        # the smallest: three requests that have just begun, small heads
        dict(name="paged_single_3", op="attention", queries="1,1,1", lens="1,17,130", page=16, heads=12, kv_heads=4,
             dim=64, causal=True, dtype="fp16"),
        # -- norms of the query and key heads with the rotary positions
        # a large batch of prompt tokens as they leave the fused QKV projection
        dict(name="qk_norm_prompt_16384", op="norm", tokens=16384, heads=32, kv_heads=8, dim=128, rot=128,
             layout="half", kind="rms", yarn=False, first=0, page=0, dtype="bf16"),
        # a prompt's chunk on its way into the pages
        dict(name="qk_norm_chunk_701", op="norm", tokens=701, heads=40, kv_heads=8, dim=128, rot=128, layout="half",
             kind="rms", yarn=True, first=31000, page=64, dtype="bf16"),
        # one token of each of 48 requests, half of each head turned
        dict(name="qk_norm_single_48", op="norm", tokens=48, heads=16, kv_heads=2, dim=64, rot=32,
             layout="interleaved", kind="layer", yarn=False, first=900, page=16, dtype="fp16"),
        # -- pages
        # holes closed in the caches of 8 layers
        dict(name="copy_pages_150", op="copy", moves=150, pages=500, caches=16, page=32, kv_heads=8, dim=128,
             dtype="bf16"),
        # a few small pages in two layers' caches
        dict(name="copy_pages_3", op="copy", moves=3, pages=40, caches=4, page=16, kv_heads=2, dim=64, dtype="fp16"),
        # one prompt continued 15 times more
        dict(name="fork_15", op="fork", forks=15, rows=40, table=64, filled=40, pages=200, caches=32, page=64,
             kv_heads=8, dim=128, one=True, dtype="bf16"),
        # beams that change places, small pages
        dict(name="fork_5", op="fork", forks=5, rows=16, table=32, filled=20, pages=500, caches=12, page=16, kv_heads=4,
             dim=128, one=False, dtype="bf16"),
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["attention"] * 5 + ["norm"] * 3 + ["copy", "fork"])
    heads, kv_heads = rng.choice([(40, 8), (32, 8), (28, 4), (16, 16), (16, 2), (12, 4), (12, 1)])
    dim = rng.choice([128, 128, 64])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "attention":
        form = rng.choice(["single", "draft", "chunk", "mixed"])
        n = _log_int(rng, 1, 64) if form != "chunk" else rng.choice([1, 1, 2, 3])
        longest = _log_int(rng, 32, max(256, min(32768, 1600000 // (n * kv_heads))))
        queries, lens = [], []
        for i in range(n):
            if form == "chunk" or (form == "mixed" and i < 2):
                q = _log_int(rng, 6, max(64, 400 // max(1, longest * n // 32768)))
            else:
                q = rng.randint(2, 8) if form == "draft" else 1
            queries.append(q)
            lens.append(q + rng.randint(0, longest))
        return dict(op=op, queries=",".join(map(str, queries)), lens=",".join(map(str, lens)),
                    page=rng.choice([16, 32, 48, 64, 128, 256]), heads=heads, kv_heads=kv_heads, dim=dim,
                    causal=rng.random() < 0.9, dtype=dtype)
    if op == "norm":
        return dict(op=op, tokens=_log_int(rng, 1, 12000), heads=heads, kv_heads=kv_heads, dim=dim,
                    rot=rng.choice([dim, dim, dim // 2]), layout=rng.choice(["half", "interleaved"]),
                    kind=rng.choice(["rms", "rms", "layer"]), yarn=rng.random() < 0.3, first=_log_int(rng, 1, 500000),
                    page=rng.choice([0, 16, 64]), dtype=dtype)
    page, caches = rng.choice([16, 32, 64]), 2 * _log_int(rng, 1, 16)
    if op == "copy":
        moves = _log_int(rng, 1, min(128, 2048 // caches))
        return dict(op=op, moves=moves, pages=2 * moves + rng.randint(0, 100), caches=caches, page=page,
                    kv_heads=rng.choice([2, 4, 8]), dim=dim, dtype=dtype)
    forks, one, filled = _log_int(rng, 1, 24), rng.random() < 0.5, rng.randint(1, 30)
    return dict(op=op, forks=forks, rows=2 * forks + rng.randint(0, 9), table=filled + rng.randint(0, 20), filled=filled,
                pages=forks + filled * (1 if one else forks) + rng.randint(0, 50), caches=caches, page=page,
                kv_heads=rng.choice([2, 4]), dim=dim, one=one, dtype=dtype)


def _numbers(text):
    return [int(x) for x in text.split(",")]


def _pages_of(n, page):
    return -(-n // page)


def work(case):
    op = case["op"]
    if op == "attention":
        queries, lens = _numbers(case["queries"]), _numbers(case["lens"])
        pairs = sum(n * m - (n * (n - 1) // 2 if case["causal"] else 0) for n, m in zip(queries, lens))
        return {"bytes": 4 * case["dim"] * (case["heads"] * sum(queries) + case["kv_heads"] * sum(lens)),
                "flops": 4 * case["dim"] * case["heads"] * pairs}
    if op == "norm":
        t, turned = case["tokens"], case["heads"] + case["kv_heads"]
        rows = turned + (case["kv_heads"] if case["page"] else 0)
        return {"bytes": 4 * t * rows * case["dim"] + 16 * t, "flops": t * turned * (4 * case["dim"] + 3 * case["rot"])}
    page = 2 * case["page"] * case["kv_heads"] * case["dim"]
    if op == "copy":
        return {"bytes": 2 * case["moves"] * case["caches"] * page, "flops": 0}
    return {"bytes": 2 * case["forks"] * case["caches"] * page + 8 * case["forks"] * case["filled"], "flops": 0}


def _frequencies(case):
    """Radians per position of each pair, in 64 bits."""
    f = 10000.0 ** -(torch.arange(0, case["rot"], 2, dtype=torch.float64) / case["rot"])
    if case["yarn"]:  # pairs that turn often keep their frequency, slow ones are interpolated
        keep = ((16384 * f / (2 * math.pi) - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        f = f * keep + f / 8.0 * (1 - keep)
    return f.to(DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]

    def normal(*shape, dtype=dt, std=1.0):
        return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)

    def shuffled(n):
        return torch.randperm(n, generator=g, device=DEV)

    op = case["op"]
    s = dict(case)
    hk, d, page = case["kv_heads"], case["dim"], case["page"]
    if op == "attention":
        queries, lens = _numbers(case["queries"]), _numbers(case["lens"])
        s["n"], s["m"] = queries, lens
        s["scale"] = d ** -0.5
        # the queries are a part of one projection's output
        s["q"] = normal(sum(queries), case["heads"] + 2 * hk, d)[:, :case["heads"]]
        used = [_pages_of(m, page) for m in lens]
        pages = sum(used) + 8
        s["k_pages"], s["v_pages"] = normal(pages, page, hk, d), normal(pages, page, hk, d)
        # pages in any order; what lies behind a sequence's last page is not used
        order = shuffled(pages).to(torch.int32)
        table = torch.zeros(len(lens), max(used) + 1, dtype=torch.int32, device=DEV)
        at = 0
        for b, u in enumerate(used):
            table[b, :u] = order[at:at + u]
            at += u
        s["table"] = table
        s["k_lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        s["cu_q"] = torch.tensor([0] + queries, device=DEV).cumsum(0).to(torch.int32)
        return s
    if op == "norm":
        t, hq = case["tokens"], case["heads"]
        qkv = normal(t, hq + 2 * hk, d, std=2.0)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        s["q_gamma"], s["k_gamma"] = ((1 + normal(d, dtype=torch.float32, std=0.2)).to(dt) for _ in range(2))
        s["freqs"] = _frequencies(case)
        s["amp"] = 0.1 * math.log(8.0) + 1.0 if case["yarn"] else 1.0
        s["positions"] = torch.arange(t, device=DEV, dtype=torch.int64) + case["first"]
        if page:  # every token has a row of its own, its sequence's pages lie in any order
            pages = _pages_of(t, page) + 3
            order = shuffled(pages)
            i = torch.arange(t, device=DEV)
            s["slots"] = order[i // page] * page + i % page
            s["k_pages"] = torch.zeros(pages, page, hk, d, dtype=dt, device=DEV)
            s["v_pages"] = torch.zeros_like(s["k_pages"])
        return s
    # every layer's K and V
    s["kv"] = [normal(case["pages"], page, hk, d) for _ in range(case["caches"])]
    order = shuffled(case["pages"]).to(torch.int32)
    if op == "copy":
        s["src"], s["dst"] = order[:case["moves"]].clone(), order[case["moves"]:2 * case["moves"]].clone()
        return s
    forks, filled = case["forks"], case["filled"]
    s["new"] = order[:forks].clone()
    rows = shuffled(case["rows"]).to(torch.int32)
    s["dst"] = rows[:forks].clone()
    s["src"] = (rows[-1:].expand(forks) if case["one"] else rows[forks:2 * forks]).clone()
    s["table"] = torch.zeros(case["rows"], case["table"], dtype=torch.int32, device=DEV)
    s["k_lens"] = torch.zeros(case["rows"], dtype=torch.int32, device=DEV)
    old = order[forks:]
    for i in range(1 if case["one"] else forks):  # sequences that end within their last page
        s["table"][s["src"][i].long(), :filled] = old[i * filled:(i + 1) * filled]
    lens = torch.randint(1, page, (forks,), generator=g, device=DEV) + (filled - 1) * page
    s["k_lens"][s["src"].long()] = (lens[:1].expand(forks) if case["one"] else lens).to(torch.int32)
    return s


# ---------------------------------------------------------------- plain forms
def _plain_attention(s):
    hq, hk, d, page = s["heads"], s["kv_heads"], s["dim"], s["page"]
    out, at = [], 0
    for b, (n, m) in enumerate(zip(s["n"], s["m"])):
        pages = s["table"][b, :_pages_of(m, page)].long()
        k = s["k_pages"][pages].view(-1, hk, d)[:m].float().permute(1, 2, 0)
        v = s["v_pages"][pages].view(-1, hk, d)[:m].float().transpose(0, 1)
        q = s["q"][at:at + n].float().view(n, hk, hq // hk, d).permute(1, 2, 0, 3).reshape(hk, -1, d)
        score = torch.matmul(q, k).mul_(s["scale"]).view(hk, hq // hk, n, m)
        if s["causal"] and n > 1:
            i, j = torch.arange(n, device=DEV), torch.arange(m, device=DEV)
            score.masked_fill_(j[None, :] > i[:, None] + (m - n), -math.inf)
        p = score.sub_(score.amax(-1, keepdim=True)).exp_()
        o = torch.matmul(p.view(hk, -1, m), v).view(hk, hq // hk, n, d) / p.sum(-1, keepdim=True)
        out.append(o.permute(2, 0, 1, 3).reshape(n, hq, d).to(s["q"].dtype))
        at += n
    return torch.cat(out)


def _plain_norm(s):
    angle = s["positions"].double()[:, None] * s["freqs"][None, :]
    c, sn = ((f(angle) * s["amp"]).float()[:, None, :] for f in (torch.cos, torch.sin))
    rot, half, out = s["rot"], s["layout"] == "half", []
    for x, gamma in ((s["q"], s["q_gamma"]), (s["k"], s["k_gamma"])):
        y = x.float()
        if s["kind"] == "layer":
            y = y - y.mean(-1, keepdim=True)
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * gamma.float()
        r, rest = y[..., :rot], y[..., rot:]
        a, b = (r[..., :rot // 2], r[..., rot // 2:]) if half else (r[..., 0::2], r[..., 1::2])
        p, q = a * c - b * sn, b * c + a * sn
        r = torch.cat([p, q], -1) if half else torch.stack([p, q], -1).flatten(-2)
        out.append(torch.cat([r, rest], -1).to(x.dtype))
    if not s["page"]:
        return tuple(out)
    s["k_pages"].flatten(0, 1)[s["slots"]] = out[1]
    s["v_pages"].flatten(0, 1)[s["slots"]] = s["v"]
    return out[0], s["k_pages"], s["v_pages"]


def _plain_copy(s):
    src, dst = s["src"].long(), s["dst"].long()
    for c in s["kv"]:
        c[dst] = c[src]
    return s["kv"]


def _plain_fork(s):
    src, dst = s["src"].long(), s["dst"].long()
    lens = s["k_lens"][src]
    last = (lens // s["page"]).long()
    rows = s["table"][src]
    page = rows.gather(1, last[:, None])[:, 0].long()
    column = torch.arange(s["table"].shape[1], device=DEV)[None, :]
    rows = torch.where(column < last[:, None], rows, s["table"][dst])
    s["table"][dst] = torch.where(column == last[:, None], s["new"][:, None], rows)
    s["k_lens"][dst] = lens
    new = s["new"].long()
    for c in s["kv"]:
        c[new] = c[page]
    return [s["table"], s["k_lens"], *s["kv"]]


def run(state):
    s = state
    if own:
        return _own(s)
    return {"attention": _plain_attention, "norm": _plain_norm, "copy": _plain_copy, "fork": _plain_fork}[s["op"]](s)


def _own(s):
    import w8a8_int8_linear_gb300 as w8
    op = s["op"]
    if op == "attention":
        return w8.paged_attention(s["q"], s["k_pages"], s["v_pages"], s["table"], s["k_lens"], cu_q=s["cu_q"],
                                  max_queries=max(s["n"]), causal=s["causal"], scale=s["scale"])
    if op == "norm":
        kind = w8.LAYER_NORM if s["kind"] == "layer" else w8.RMS_NORM
        if not s["page"]:
            return w8.qk_norm_rotary(s["q"], s["k"], s["positions"], s["freqs"], q_gamma=s["q_gamma"],
                                     k_gamma=s["k_gamma"], kind=kind, layout=s["layout"], amplitude=s["amp"])
        q = w8.qk_norm_rotary_append(s["q"], s["k"], s["v"], s["positions"], s["freqs"], s["k_pages"], s["v_pages"],
                                     s["slots"], q_gamma=s["q_gamma"], k_gamma=s["k_gamma"], kind=kind,
                                     layout=s["layout"], amplitude=s["amp"])
        return q, s["k_pages"], s["v_pages"]
    if op == "copy":
        w8.copy_pages(s["kv"], s["src"], s["dst"])
        return s["kv"]
    w8.fork_sequences(s["kv"], s["table"], s["k_lens"], s["src"], s["dst"], s["new"], page_size=s["page"])
    return [s["table"], s["k_lens"], *s["kv"]]


# ---------------------------------------------------------------- definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "attention":
        return _exact_attention(case, s)
    if op == "norm":
        turn = torch.polar(torch.full((case["tokens"], case["rot"] // 2), float(s["amp"]), dtype=torch.float64,
                                      device=DEV), torch.outer(s["positions"].double(), s["freqs"]))
        n, out = case["rot"] // 2, []
        for x, gamma in ((s["q"], s["q_gamma"]), (s["k"], s["k_gamma"])):
            y = x.double()
            if case["kind"] == "layer":
                y = y - y.sum(2, keepdim=True) / case["dim"]
            y = y / torch.sqrt((y * y).sum(2, keepdim=True) / case["dim"] + 1e-6) * gamma.double()
            first, second = (slice(0, n), slice(n, 2 * n)) if case["layout"] == "half" else (
                slice(0, 2 * n, 2), slice(1, 2 * n, 2))
            z = torch.complex(y[..., first].clone(), y[..., second].clone()) * turn[:, None, :]
            y[..., first], y[..., second] = z.real, z.imag
            out.append(y)
        if not case["page"]:
            return tuple(out)
        caches = []
        for new, cache in ((out[1], s["k_pages"]), (s["v"].double(), s["v_pages"])):
            cache = cache.double()
            cache[s["slots"] // case["page"], s["slots"] % case["page"]] = new
            caches.append(cache)
        return out[0], *caches
    # (the pairs one after another, as numbers of the host)
    kv = [c.double() for c in s["kv"]]
    src, dst = s["src"].tolist(), s["dst"].tolist()
    if op == "copy":
        for a, b in zip(src, dst):
            for c in kv:
                c[b] = c[a]
        return kv
    table, lens, new = s["table"].tolist(), s["k_lens"].tolist(), s["new"].tolist()
    for a, b, page in zip(src, dst, new):
        lens[b] = lens[a]
        full = lens[a] // case["page"]
        for c in kv:
            c[page] = c[table[a][full]]
        table[b][:full + 1] = table[a][:full] + [page]
    return [torch.tensor(table, dtype=torch.int32, device=DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), *kv]


def _exact_attention(case, s):
    group = case["heads"] // case["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    at = 0
    for b, (n, m) in enumerate(zip(s["n"], s["m"])):
        key = torch.arange(m, device=DEV)
        row = s["table"][b].long()[key // case["page"]] * case["page"] + key % case["page"]
        hidden = None
        if case["causal"]:
            hidden = torch.ones(n, m, dtype=torch.bool, device=DEV).tril(m - n).logical_not()
        for h in range(case["kv_heads"]):
            k = s["k_pages"][:, :, h].flatten(0, 1).index_select(0, row).double()
            v = s["v_pages"][:, :, h].flatten(0, 1).index_select(0, row).double()
            heads = slice(h * group, (h + 1) * group)
            score = (s["q"][at:at + n, heads].double().transpose(0, 1) @ k.T) * s["scale"]
            if hidden is not None:
                score = score.masked_fill(hidden, -math.inf)
            out[at:at + n, heads] = (torch.softmax(score, -1) @ v).transpose(0, 1)
        at += n
    return out
