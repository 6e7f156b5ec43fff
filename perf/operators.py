"""Measured cases of the operators between a W8A8 transformer layer's Linears.

Three operators: `attention` (packed prompts, and few queries over a cache),
`rotary` / `rotary_append` (rotary positions, and the cache rows written with
them) and `residual_norm_quant` (branch norm, gate, residual, next norm,
quantization).  `run` computes a case in plain 32-bit torch operations, or,
where `own` is true, with the package's entry points.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # -- attention over prompts
        # one long prompt, grouped heads of a 5120-wide model, causal
        dict(name="prompt_8192", op="prompt", lens="8192", heads=40, kv_heads=8, dim=128, causal=True, dtype="bf16"),
        # a batch of requests of very different lengths packed without padding, 4096-wide model
        dict(name="prompt_packed_ragged", op="prompt", lens="2048,1000,257,77,1,1531", heads=32, kv_heads=8, dim=128,
             causal=True, dtype="bf16"),
        # full (not causal) attention over image or video tokens, ungrouped heads of 64
        dict(name="full_4096_d64", op="prompt", lens="4096", heads=32, kv_heads=32, dim=64, causal=False,
             dtype="fp16"),
        # -- attention of single tokens over a cache
        # the smallest: four requests that have just begun
        dict(name="decode_4_short", op="decode", lens="513,300,77,128", capacity=640, queries=1, heads=32, kv_heads=8,
             dim=128, dtype="bf16"),
        # a serving batch in full swing, ragged lengths
        dict(name="decode_64_ragged", op="decode", lens=",".join(str(1 + (i * 2654435761) % 4096) for i in range(64)),
             capacity=4096, queries=1, heads=40, kv_heads=8, dim=128, dtype="bf16"),
        # two requests over very long caches, where the work has to be split along the keys
        dict(name="decode_2_long", op="decode", lens="131072,99991", capacity=131072, queries=1, heads=32, kv_heads=8,
             dim=128, dtype="bf16"),
        # -- rotary positions
        # Q and K of a large batch of prompt tokens, as they leave the fused QKV projection
        dict(name="rotary_prompt_32768", op="rotary", tokens=32768, heads=40, kv_heads=8, dim=128, rot=128,
             layout="half", scaling="plain", first=0, dtype="bf16"),
        # part of the head, interleaved, an odd number of tokens of a long context
        dict(name="rotary_part_1000", op="rotary", tokens=1000, heads=32, kv_heads=32, dim=64, rot=32,
             layout="interleaved", scaling="linear", first=100000, dtype="fp16"),
        # one token for each of 64 requests, K and V written to their cache rows
        dict(name="rotary_append_64", op="append", tokens=64, capacity=512, heads=40, kv_heads=8, dim=128, rot=128,
             layout="half", scaling="yarn", first=131000, dtype="bf16"),
        # -- residual, norm and quantization
        # between attention and FFN of a 5120-wide model, large prompt batch, on to the next W8A8 Linear
        dict(name="norm_prompt_32768", op="norm", rows=32768, width=5120, kind="rms", groups=0, branch=False,
             residual="bf16", alpha=1.0, out="image"),
        # gated and modulated blocks (gate, scale and shift per sample), fp32 residual stream
        dict(name="norm_modulated_4096", op="norm", rows=4096, width=4096, kind="layer", groups=2, branch=False,
             residual="fp32", alpha=1.0, out="y"),
        # single tokens, norms before and after the block, scaled residual
        dict(name="norm_4_branch", op="norm", rows=4, width=5120, kind="rms", groups=0, branch=True, residual="bf16",
             alpha=0.5, out="y"),
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "decode", "decode", "rotary", "append", "norm", "norm"])
    heads, kv_heads = rng.choice([(40, 8), (32, 8), (32, 32), (16, 2), (28, 4), (12, 1)])
    dim = rng.choice([128, 128, 64])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "prompt":
        n = rng.choice([1, 1, 2, 4, 8])
        lens = [_log_int(rng, 16, 5700)] if n == 1 else [_log_int(rng, 1, 2048) for _ in range(n)]
        return dict(op=op, lens=",".join(map(str, lens)), heads=heads, kv_heads=kv_heads, dim=dim,
                    causal=rng.random() < 0.7, dtype=dtype)
    if op == "decode":
        n = _log_int(rng, 1, 96)
        longest = _log_int(rng, 64, max(256, min(131072, 262144 // n)))
        lens = [max(4, rng.randint(longest // 4, longest)) for _ in range(n)]
        return dict(op=op, lens=",".join(map(str, lens)), capacity=longest + rng.randint(1, 64),
                    queries=rng.choice([1, 1, 1, 2, 4]), heads=heads, kv_heads=kv_heads if heads != kv_heads else 8,
                    dim=dim, dtype=dtype)
    if op in ("rotary", "append"):
        rot = rng.choice([dim, dim, dim // 2])
        case = dict(op=op, tokens=_log_int(rng, 1, 16384 if op == "rotary" else 256), heads=heads, kv_heads=kv_heads,
                    dim=dim, rot=rot, layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["plain", "linear", "ntk", "yarn"]), first=_log_int(rng, 1, 1000000),
                    dtype=dtype)
        if op == "append":
            case["capacity"] = _log_int(rng, 16, 512)
        return case
    width = 8 * _log_int(rng, 64, 1728)
    return dict(op=op, rows=_log_int(rng, 1, min(16384, 100000000 // width)), width=width,
                kind=rng.choice(["rms", "layer"]), groups=rng.choice([0, 0, 1, 2, 3]), branch=rng.random() < 0.3,
                residual=rng.choice(["bf16", "fp32"]), alpha=rng.choice([1.0, 1.0, 0.5]),
                out=rng.choice(["image", "y", "codes"]))


def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


def work(case):
    op = case["op"]
    if op in ("prompt", "decode"):
        k_lens = _lens(case)
        q_lens = k_lens if op == "prompt" else [case["queries"]] * len(k_lens)
        causal = case.get("causal", True)
        pairs = sum(n * m - (n * (n - 1) // 2 if causal else 0) for n, m in zip(q_lens, k_lens))
        bytes_ = 2 * case["dim"] * (2 * case["heads"] * sum(q_lens) + 2 * case["kv_heads"] * sum(k_lens))
        return {"bytes": bytes_, "flops": 4 * case["dim"] * case["heads"] * pairs}
    if op in ("rotary", "append"):
        t, rows = case["tokens"], case["heads"] + case["kv_heads"] * (2 if op == "append" else 1)
        return {"bytes": 4 * t * rows * case["dim"] + 8 * t + 4 * case["rot"],
                "flops": 3 * t * (case["heads"] + case["kv_heads"]) * case["rot"]}
    m, k = case["rows"], case["width"]
    res = 4 if case["residual"] == "fp32" else 2
    out = {"image": 2 * k + 4, "y": 2 * k, "codes": k + 4}[case["out"]]
    return {"bytes": m * (2 * k + 2 * res * k + out) + 2 * k * (1 + 3 * case["groups"]), "flops": 12 * m * k}


def _frequencies(case):
    """Radians per position of each pair, in 64 bits."""
    r, base, factor = case["rot"], 10000.0, 8.0
    i = torch.arange(0, r, 2, dtype=torch.float64) / r
    if case["scaling"] == "ntk":
        base *= factor ** (r / (r - 2))
    f = base ** -i
    if case["scaling"] == "linear":
        f = f / factor
    if case["scaling"] == "yarn":  # pairs that turn often keep their frequency, slow ones are interpolated
        turns = 16384 * f / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        f = f * keep + f / factor * (1 - keep)
    return f.to(DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))

    def normal(*shape, dtype=torch.bfloat16, std=1.0):
        return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)

    op = case["op"]
    s = dict(case)
    if op in ("prompt", "decode"):
        dt = DTYPES[case["dtype"]]
        hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
        lens = _lens(case)
        s["scale"] = d ** -0.5
        if op == "prompt":  # Q, K and V are the parts of one projection's output
            qkv = normal(sum(lens), hq + 2 * hk, d, dtype=dt)
            s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
            s["cu"] = torch.tensor([0] + lens, device=DEV).cumsum(0).to(torch.int32)
            s["longest"] = max(lens)
        else:
            n, cap = len(lens), case["capacity"]
            s["q"] = normal(n * case["queries"], hq, d, dtype=dt)
            s["k"], s["v"] = normal(n * cap, hk, d, dtype=dt), normal(n * cap, hk, d, dtype=dt)
            s["k_lens"] = torch.tensor(lens, device=DEV, dtype=torch.int32)
        return s
    if op in ("rotary", "append"):
        dt = DTYPES[case["dtype"]]
        t, hq, hk, d = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
        qkv = normal(t, hq + 2 * hk, d, dtype=dt)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        s["freqs"] = _frequencies(case)
        s["amp"] = 0.1 * math.log(8.0) + 1.0 if case["scaling"] == "yarn" else 1.0
        if op == "rotary":
            s["positions"] = torch.arange(t, device=DEV, dtype=torch.int64) + case["first"]
        else:  # every request is at a place of its own
            cap = case["capacity"]
            at = torch.randint(0, cap, (t,), generator=g, device=DEV)
            s["positions"] = at + case["first"]
            s["slots"] = torch.arange(t, device=DEV, dtype=torch.int64) * cap + at
            s["k_cache"] = torch.zeros(t * cap, hk, d, dtype=dt, device=DEV)
            s["v_cache"] = torch.zeros_like(s["k_cache"])
        return s
    m, k = case["rows"], case["width"]
    s["x"] = normal(m, k, dtype=DTYPES[case["residual"]], std=2.0)
    s["b"] = normal(m, k)
    s["gamma"] = (1 + normal(k, dtype=torch.float32, std=0.1)).to(torch.bfloat16)
    s["branch_gamma"] = (1 + normal(k, dtype=torch.float32, std=0.1)).to(torch.bfloat16) if case["branch"] else None
    s["gate"] = s["mod_scale"] = s["mod_shift"] = None
    if case["groups"]:  # the modulation of each sample, as it leaves its projection
        s["gate"], s["mod_scale"], s["mod_shift"] = normal(case["groups"], 3 * k, std=0.3).chunk(3, dim=1)
    s["rows_per_group"] = -(-m // max(1, case["groups"]))
    return s


# ---------------------------------------------------------------- plain forms
def _plain_attention(q, k, v, q_at, q_ok, k_at, k_ok, offset, scale, causal):
    """q_at / k_at [B, n] / [B, m]: the packed rows of each sequence, padded
    (q_ok / k_ok false); query i of sequence b sees keys j <= i + offset[b]."""
    hq, hk, d = q.shape[1], k.shape[1], q.shape[2]
    b, n = q_at.shape
    m = k_at.shape[1]
    qf = q[q_at].float().view(b, n, hk, hq // hk, d).permute(0, 2, 3, 1, 4).reshape(b, hk, -1, d)
    kf = k[k_at].float().permute(0, 2, 3, 1)
    vf = v[k_at].float().permute(0, 2, 1, 3)
    see = k_ok[:, None, :].expand(b, n, m)
    if causal:
        i, j = torch.arange(n, device=q.device), torch.arange(m, device=q.device)
        see = see & (j[None, None, :] <= i[None, :, None] + offset[:, None, None])
    s = torch.matmul(qf, kf).mul_(scale).view(b, hk, hq // hk, n, m)
    s.masked_fill_(~see[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(b, hk, -1, m), vf).view(b, hk, hq // hk, n, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    o = o.permute(0, 3, 1, 2, 4).reshape(b, n, hq, d).to(q.dtype)
    out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    out[q_at[q_ok]] = o[q_ok]
    return out


def _plain_prompt(s):
    start = s["cu"][:-1].long()
    lens = s["cu"][1:].long() - start
    j = torch.arange(s["longest"], device=DEV)
    ok = j[None, :] < lens[:, None]
    at = torch.where(ok, start[:, None] + j[None, :], torch.zeros_like(start)[:, None])
    return _plain_attention(s["q"], s["k"], s["v"], at, ok, at, ok, torch.zeros_like(lens), s["scale"], s["causal"])


def _plain_decode(s):
    lens = s["k_lens"].long()
    n, nq, cap = lens.numel(), s["queries"], s["capacity"]
    q_at = torch.arange(n * nq, device=DEV).view(n, nq)
    j = torch.arange(cap, device=DEV)
    k_at = torch.arange(n, device=DEV)[:, None] * cap + j[None, :]
    return _plain_attention(s["q"], s["k"], s["v"], q_at, torch.ones_like(q_at, dtype=torch.bool), k_at,
                            j[None, :] < lens[:, None], lens - nq, s["scale"], True)


def _plain_rotate(x, c, sn, rot, layout):
    y = x.float()
    r, rest = y[..., :rot], y[..., rot:]
    a, b = (r[..., :rot // 2], r[..., rot // 2:]) if layout == "half" else (r[..., 0::2], r[..., 1::2])
    p, q = a * c - b * sn, b * c + a * sn
    r = torch.cat([p, q], -1) if layout == "half" else torch.stack([p, q], -1).flatten(-2)
    return torch.cat([r, rest], -1).to(x.dtype)


def _plain_rotary(s):
    angle = s["positions"].double()[:, None] * s["freqs"][None, :]
    c, sn = ((f(angle) * s["amp"]).float()[:, None, :] for f in (torch.cos, torch.sin))
    return tuple(_plain_rotate(x, c, sn, s["rot"], s["layout"]) for x in (s["q"], s["k"]))


def _plain_norm(s):
    h = s["b"].float()
    if s["branch_gamma"] is not None:
        h = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6) * s["branch_gamma"].float()
    row = torch.arange(s["rows"], device=DEV) // s["rows_per_group"]
    if s["gate"] is not None:
        h = h * s["gate"].float()[row]
    h = s["x"].float() * s["alpha"] + h
    d = h - h.mean(-1, keepdim=True) if s["kind"] == "layer" else h
    y = d * torch.rsqrt(d.square().mean(-1, keepdim=True) + 1e-6) * s["gamma"].float()
    if s["mod_scale"] is not None:
        y = y * (1 + s["mod_scale"].float()[row]) + s["mod_shift"].float()[row]
    h = h.to(s["x"].dtype)
    if s["out"] == "y":
        return h, y.to(torch.bfloat16)
    sx = y.abs().amax(-1) / 127
    q = (y / sx[:, None]).round().clamp(-127, 127)
    if s["out"] == "image":
        return h, q.to(torch.bfloat16), sx
    return h, (q * sx[:, None]).to(torch.bfloat16), sx


def run(state):
    s, op = state, state["op"]
    if own:
        return _own(s, op)
    if op == "prompt":
        return _plain_prompt(s)
    if op == "decode":
        return _plain_decode(s)
    if op == "rotary":
        return _plain_rotary(s)
    if op == "append":
        q, k = _plain_rotary(s)
        s["k_cache"][s["slots"]] = k
        s["v_cache"][s["slots"]] = s["v"]
        return q, s["k_cache"], s["v_cache"]
    return _plain_norm(s)


def _own(s, op):
    import w8a8_int8_linear_gb300 as w8
    if op == "prompt":
        return w8.attention(s["q"], s["k"], s["v"], cu_q=s["cu"], cu_k=s["cu"], causal=s["causal"], scale=s["scale"])
    if op == "decode":
        return w8.attention(s["q"], s["k"], s["v"], k_lens=s["k_lens"], batch=s["k_lens"].numel(), scale=s["scale"])
    if op == "rotary":
        return w8.rotary(s["q"], s["k"], s["positions"], s["freqs"], layout=s["layout"], amplitude=s["amp"])
    if op == "append":
        q = w8.rotary_append(s["q"], s["k"], s["v"], s["positions"], s["freqs"], s["k_cache"], s["v_cache"],
                             s["slots"], layout=s["layout"], amplitude=s["amp"])
        return q, s["k_cache"], s["v_cache"]
    out = s["out"]
    h, img, sx, xq, y = w8.residual_norm_quant(
        s["x"], s["b"], gamma=s["gamma"], eps=1e-6, kind=w8.LAYER_NORM if s["kind"] == "layer" else w8.RMS_NORM,
        alpha=s["alpha"], branch_gamma=s["branch_gamma"], gate=s["gate"], mod_scale=s["mod_scale"],
        mod_shift=s["mod_shift"], rows_per_group=s["rows_per_group"], image=out == "image", codes=out == "codes",
        y=out == "y")
    if out == "y":
        return h, y
    if out == "image":
        return h, img, sx
    return h, (xq.float() * sx[:, None]).to(torch.bfloat16), sx


# ---------------------------------------------------------------- definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("prompt", "decode"):
        return _exact_attention(case, s)
    if op in ("rotary", "append"):
        out = []
        turn = torch.polar(torch.full((case["tokens"], case["rot"] // 2), float(s["amp"]), dtype=torch.float64,
                                      device=DEV), torch.outer(s["positions"].double(), s["freqs"]))
        for x in (s["q"], s["k"]):
            y = x.double().clone()
            if case["layout"] == "half":
                z = torch.complex(y[..., :case["rot"] // 2].clone(), y[..., case["rot"] // 2:case["rot"]].clone())
            else:
                z = torch.complex(y[..., 0:case["rot"]:2].clone(), y[..., 1:case["rot"]:2].clone())
            z = z * turn[:, None, :]
            if case["layout"] == "half":
                y[..., :case["rot"] // 2], y[..., case["rot"] // 2:case["rot"]] = z.real, z.imag
            else:
                y[..., 0:case["rot"]:2], y[..., 1:case["rot"]:2] = z.real, z.imag
            out.append(y)
        if op == "rotary":
            return tuple(out)
        k_cache = torch.zeros(s["k_cache"].shape, dtype=torch.float64, device=DEV)
        v_cache = torch.zeros_like(k_cache)
        k_cache[s["slots"]], v_cache[s["slots"]] = out[1], s["v"].double()
        return out[0], k_cache, v_cache
    m, k = case["rows"], case["width"]
    hs, ys = [], []
    for at in range(0, m, 4096):
        rows = slice(at, min(m, at + 4096))
        b = s["b"][rows].double()
        if s["branch_gamma"] is not None:
            b = b / torch.sqrt((b * b).sum(1, keepdim=True) / k + 1e-6) * s["branch_gamma"].double()
        group = torch.div(torch.arange(rows.start, rows.stop, device=DEV), s["rows_per_group"], rounding_mode="floor")
        if s["gate"] is not None:
            b = b * s["gate"].double().index_select(0, group)
        h = case["alpha"] * s["x"][rows].double() + b
        c = h
        if case["kind"] == "layer":
            c = h - h.sum(1, keepdim=True) / k
        y = c / torch.sqrt((c * c).sum(1, keepdim=True) / k + 1e-6) * s["gamma"].double()
        if s["mod_scale"] is not None:
            y = y + y * s["mod_scale"].double().index_select(0, group) + s["mod_shift"].double().index_select(0, group)
        hs.append(h)
        ys.append(y)
    h, y = torch.cat(hs), torch.cat(ys)
    if case["out"] == "y":
        return h, y
    sx = y.abs().max(1).values / 127.0
    q = torch.round(y / sx[:, None])
    return (h, q if case["out"] == "image" else q * sx[:, None], sx)


def _exact_attention(case, s):
    hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
    group = hq // hk
    lens = _lens(case)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    q_at = 0
    for b, m in enumerate(lens):
        n = m if case["op"] == "prompt" else case["queries"]
        k_at = q_at if case["op"] == "prompt" else b * case["capacity"]
        hidden = None
        if case.get("causal", True):
            hidden = torch.ones(n, m, dtype=torch.bool, device=DEV).tril(m - n).logical_not()
        for h in range(hk):
            k = s["k"][k_at:k_at + m, h].double()
            v = s["v"][k_at:k_at + m, h].double()
            q = s["q"][q_at:q_at + n, h * group:(h + 1) * group].double().transpose(0, 1)
            score = (q @ k.T) * s["scale"]
            if hidden is not None:
                score = score.masked_fill(hidden, -math.inf)
            out[q_at:q_at + n, h * group:(h + 1) * group] = (torch.softmax(score, -1) @ v).transpose(0, 1)
        q_at += n
    return out
