"""The operators between a transformer layer's W8A8 Linears.

`attention` (packed prompts, and few queries over a cache), `rotary` and
`rotary_append` (rotary positions, and the cache rows written with them) and
`residual_norm_quant` (branch norm, gate, residual, next norm, modulation and
int8 quantization in one pass).  As in the rest of the binding a function
only checks its tensors, allocates outputs and passes pointers, sizes and the
current stream to the library (include/w8a8.h states the arithmetic); nothing
synchronizes, so every call can be captured into a CUDA graph.
"""
import math

import torch
from torch._C import _cuda_getCurrentRawStream as _raw_stream

from . import RMS_NORM, _check, lib

HALF = "half"
INTERLEAVED = "interleaved"

_DTYPE = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_LAYOUT = {HALF: 0, INTERLEAVED: 1}


def _heads(t, name, dtype=None):
    """Checks a [tokens, heads, dim] tensor: on the GPU, 16-bit (of `dtype`),
    dense last dimension.  Returns its token and head strides; a dimension of
    one row has no stride of its own and gets the row length."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        if dtype is not None:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if t.dtype is not torch.bfloat16 and t.dtype is not torch.float16:
            raise TypeError(f"{name} must be torch.bfloat16 or torch.float16, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    strides = t.stride()
    if len(strides) != 3:
        raise ValueError(f"{name} must be [tokens, heads, dim]")
    token, head, last = strides
    tokens, heads, dim = t.shape
    if last != 1 and dim != 1:
        raise ValueError(f"{name} must be dense in its last dimension")
    return (token if tokens != 1 else heads * dim), (head if heads != 1 else dim)


def _indices(t, dtype, n, name):
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype:
        raise TypeError(f"{name} must be a {dtype} tensor")
    if not t.is_cuda or t.dim() != 1 or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a dense CUDA tensor of {n} values")
    return t.data_ptr()


_attention_ws = {}


def attention_workspace(device=None):
    """A workspace for `attention`, for one stream at a time (the counters at
    its start are, and stay between calls, zero)."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    ws = torch.empty(lib().w8a8_attention_workspace_size(), dtype=torch.uint8, device=device)
    ws[:lib().w8a8_attention_workspace_zeroed()].zero_()
    return ws


def _workspace_of(device, stream):
    if torch.cuda.is_current_stream_capturing():
        return attention_workspace(device)  # the graph's own, zeroed by every replay
    ws = _attention_ws.get((device.index, stream))
    if ws is None:
        ws = _attention_ws[device.index, stream] = attention_workspace(device)
    return ws


def attention(Q, K, V, cu_q=None, cu_k=None, k_lens=None, batch=1, causal=True, scale=None, out=None, lse=False,
              workspace=None):
    """softmax(scale Q K^T) V per sequence, query heads in groups over the KV
    heads; bf16 or fp16.

    Q [Tq, Hq, D], K and V [Tk, Hk, D]: the sequences' rows one after another
    (views with token and head strides are fine: parts of a fused projection,
    a cache).  cu_q / cu_k: int32 [B + 1] first rows of the sequences on the
    GPU; without them the rows are `batch` equal parts.  k_lens: int32 [B]
    keys in use of each sequence's part (a cache [B * capacity, Hk, D] that is
    filled to different lengths).  With `causal` the last query of a sequence
    sees all of its keys, the one before all but the last, and so on; a query
    that sees none gets zeros (lse: -inf).  scale: D ** -0.5.

    Returns O [Tq, Hq, D], or (O, lse fp32 [Tq, Hq]) with lse=True.  The
    workspace (`attention_workspace()`) is by default one per stream, and one
    of its own for a captured call."""
    q_token, q_head = _heads(Q, "Q")
    dtype, device = Q.dtype, Q.device
    k_token, k_head = _heads(K, "K", dtype)
    v_token, v_head = _heads(V, "V", dtype)
    if not (q_token and q_head and k_token and k_head and v_token and v_head):
        # a broadcast dimension is laid out
        Q, K, V = Q.contiguous(), K.contiguous(), V.contiguous()
        (q_token, q_head), (k_token, k_head), (v_token, v_head) = _heads(Q, "Q"), _heads(K, "K"), _heads(V, "V")
    tq, hq, d = Q.shape
    tk, hk, dk = K.shape
    if dk != d or V.shape != K.shape:
        raise ValueError("K and V must be [keys, KV heads, dim] with the queries' dim")
    if cu_q is not None:
        batch = cu_q.numel() - 1
    elif cu_k is not None:
        batch = cu_k.numel() - 1
    pq = None if cu_q is None else _indices(cu_q, torch.int32, batch + 1, "cu_q")
    pk = None if cu_k is None else _indices(cu_k, torch.int32, batch + 1, "cu_k")
    pl = None if k_lens is None else _indices(k_lens, torch.int32, batch, "k_lens")
    if out is None:
        out = torch.empty((tq, hq, d), dtype=dtype, device=device)
        o_token, o_head = hq * d, d
    else:
        o_token, o_head = _heads(out, "out", dtype)
        if out.shape != Q.shape:
            raise ValueError("out must have the shape of Q")
    stats = torch.empty((tq, hq), dtype=torch.float32, device=device) if lse else None
    stream = _raw_stream(device.index)
    ws = _workspace_of(device, stream) if workspace is None else workspace
    _check("w8a8_attention", lib().w8a8_attention(
        Q.data_ptr(), K.data_ptr(), V.data_ptr(), out.data_ptr(), None if stats is None else stats.data_ptr(), pq, pk,
        pl, _DTYPE[dtype], batch, tq, tk, hq, hk, d, q_token, q_head, k_token, k_head, v_token, v_head, o_token,
        o_head, d ** -0.5 if scale is None else scale, causal, ws.data_ptr(), ws.numel(), stream))
    return (out, stats) if lse else out


def rotary_frequencies(rot_dim, base=10000.0, scaling=None, factor=1.0, original_length=None, fast=32.0, slow=1.0,
                       device="cuda"):
    """Radians per position of each of the rot_dim / 2 pairs, fp64 [rot_dim / 2]:
    base ** (-2 k / rot_dim), for a context `factor` times longer than trained:
      "linear": all divided by factor;
      "ntk":    base * factor ** (rot_dim / (rot_dim - 2)), which divides the
                slowest pair's frequency by factor and leaves the fastest;
      "yarn":   (Peng et al. 2023) pairs that turn more than `fast` times in
                original_length positions are kept, those below `slow` turns
                divided by factor, linearly in between; used with the
                amplitude rotary_amplitude(factor) = 0.1 ln(factor) + 1."""
    if rot_dim <= 0 or rot_dim % 2:
        raise ValueError("rot_dim must be even and positive")
    if scaling not in (None, "linear", "ntk", "yarn"):
        raise ValueError("scaling must be None, 'linear', 'ntk' or 'yarn'")
    if not factor >= 1.0:
        raise ValueError("factor must be at least 1")
    k = torch.arange(0, rot_dim, 2, dtype=torch.float64) / rot_dim
    if scaling == "ntk":
        if rot_dim < 4:
            raise ValueError("'ntk' needs two pairs at least")
        base = base * factor ** (rot_dim / (rot_dim - 2))
    f = base ** -k
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        if original_length is None or not fast > slow:
            raise ValueError("'yarn' needs original_length, and fast > slow")
        keep = ((original_length * f / (2 * math.pi) - slow) / (fast - slow)).clamp(0, 1)
        f = f * keep + f / factor * (1 - keep)
    return f.to(device)


def rotary_amplitude(factor):
    """The amplitude that goes with "yarn" frequencies."""
    return 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0


def _rotary_common(Q, K, positions, freqs, layout):
    if layout not in _LAYOUT:
        raise ValueError("layout must be 'half' or 'interleaved'")
    t, hq, d = Q.shape
    if K is not None and (K.shape[0] != t or K.shape[2] != d):
        raise ValueError("K must have the tokens and the dim of Q")
    pp = _indices(positions, torch.int64, t, "positions")
    pf = _indices(freqs, torch.float64, freqs.numel(), "freqs")
    return t, hq, d, pp, pf, 2 * freqs.numel()


def rotary(Q, K, positions, freqs, layout=HALF, amplitude=1.0, inverse=False, q_out=None, k_out=None):
    """Rotary positions of Q [T, Hq, D] and K [T, Hk, D] (or None): the first
    2 * len(freqs) elements of each head turn by positions[t] * freqs[k]
    (int64 [T], fp64 from `rotary_frequencies`), the rest is copied.  Returns
    (Q', K'), new tensors unless q_out / k_out are given; these may be Q and K
    themselves.  inverse=True turns back (also the gradient's direction, at
    amplitude 1)."""
    q_token, q_head = _heads(Q, "Q")
    dtype, device = Q.dtype, Q.device
    t, hq, d, pp, pf, rot = _rotary_common(Q, K, positions, freqs, layout)
    hk = k_token = k_head = ko_token = ko_head = 0
    if K is not None:
        hk = K.shape[1]
        k_token, k_head = _heads(K, "K", dtype)
        if k_out is None:
            k_out = torch.empty((t, hk, d), dtype=dtype, device=device)
            ko_token, ko_head = hk * d, d
        else:
            ko_token, ko_head = _heads(k_out, "k_out", dtype)
            if k_out.shape != K.shape:
                raise ValueError("k_out must have the shape of K")
    if q_out is None:
        q_out = torch.empty((t, hq, d), dtype=dtype, device=device)
        qo_token, qo_head = hq * d, d
    else:
        qo_token, qo_head = _heads(q_out, "q_out", dtype)
        if q_out.shape != Q.shape:
            raise ValueError("q_out must have the shape of Q")
    _check("w8a8_rotary", lib().w8a8_rotary(
        Q.data_ptr(), None if K is None else K.data_ptr(), q_out.data_ptr(), None if K is None else k_out.data_ptr(),
        _DTYPE[dtype], t, hq, hk, d, rot, q_token, q_head, k_token, k_head, qo_token, qo_head, ko_token, ko_head,
        pp, pf, amplitude, _LAYOUT[layout], inverse, _raw_stream(device.index)))
    return q_out, (None if K is None else k_out)


def rotary_append(Q, K, V, positions, freqs, k_cache, v_cache, slots, layout=HALF, amplitude=1.0, q_out=None):
    """`rotary` for tokens that join a cache: turns Q and K, and writes K and V
    of token t to row slots[t] (int64 [T]) of k_cache / v_cache [rows, Hk, D];
    a slot outside the cache (-1 for a padding token) stores nothing.  Returns
    the turned Q."""
    q_token, q_head = _heads(Q, "Q")
    dtype, device = Q.dtype, Q.device
    k_token, k_head = _heads(K, "K", dtype)
    v_token, v_head = _heads(V, "V", dtype)
    kc_token, kc_head = _heads(k_cache, "k_cache", dtype)
    vc_token, vc_head = _heads(v_cache, "v_cache", dtype)
    t, hq, d, pp, pf, rot = _rotary_common(Q, K, positions, freqs, layout)
    hk = K.shape[1]
    if V.shape != K.shape or k_cache.shape[1:] != K.shape[1:] or v_cache.shape != k_cache.shape:
        raise ValueError("V must have the shape of K, and both caches its heads and dim")
    ps = _indices(slots, torch.int64, t, "slots")
    if q_out is None:
        q_out = torch.empty((t, hq, d), dtype=dtype, device=device)
        qo_token, qo_head = hq * d, d
    else:
        qo_token, qo_head = _heads(q_out, "q_out", dtype)
        if q_out.shape != Q.shape:
            raise ValueError("q_out must have the shape of Q")
    _check("w8a8_rotary_append", lib().w8a8_rotary_append(
        Q.data_ptr(), K.data_ptr(), V.data_ptr(), q_out.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
        _DTYPE[dtype], t, hq, hk, d, rot, k_cache.shape[0], q_token, q_head, k_token, k_head, v_token, v_head,
        qo_token, qo_head, kc_token, kc_head, vc_token, vc_head, pp, ps, pf, amplitude, _LAYOUT[layout],
        _raw_stream(device.index)))
    return q_out


def _rows(t, name, dtype, shape):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda or not t.is_contiguous() or t.shape != shape:
        raise ValueError(f"{name} must be a dense CUDA tensor of shape {tuple(shape)}")
    return t.data_ptr()


def _modulation(tensors, k, m, rows_per_group):
    """Pointers of gate, mod_scale and mod_shift ([groups, k] or [k]) and the
    row stride that they share."""
    pointers, strides = [], set()
    for t, name in zip(tensors, ("gate", "mod_scale", "mod_shift")):
        if t is None:
            pointers.append(None)
            continue
        if not isinstance(t, torch.Tensor) or t.dtype is not torch.bfloat16 or not t.is_cuda:
            raise TypeError(f"{name} must be a torch.bfloat16 CUDA tensor")
        if t.dim() == 1:
            t = t.unsqueeze(0)
        if t.dim() != 2 or t.shape[1] != k or (k != 1 and t.stride(1) != 1):
            raise ValueError(f"{name} must be [groups, {k}], dense in its last dimension")
        groups = t.shape[0]
        if groups * rows_per_group < m and not (groups == 1 and rows_per_group == 0):
            raise ValueError(f"{name} has {groups} rows of {rows_per_group} tokens each, too few for {m} tokens")
        # a single row serves every token, and its stride is not used
        if rows_per_group and m > rows_per_group:
            strides.add(t.stride(0))
        pointers.append(t.data_ptr())
    if len(strides) > 1:
        raise ValueError("gate, mod_scale and mod_shift must have the same row stride")
    return pointers, strides.pop() if strides else 0


def residual_norm_quant(X, B, gamma=None, beta=None, eps=1e-6, kind=RMS_NORM, alpha=1.0, gate=None, branch_gamma=None,
                        mod_scale=None, mod_shift=None, rows_per_group=0, h_out=None, image=True, codes=False,
                        y=False):
    """From a block's output to the next block's W8A8 Linear in one pass:

        h = alpha * X + gate * (RMSNorm(B) * branch_gamma, or B)
        y = norm(h) * gamma + beta, then y * (1 + mod_scale) + mod_shift

    X [M, K] the residual stream (bf16 or fp32), B [M, K] bf16 the branch;
    gamma, beta, branch_gamma bf16 [K]; gate, mod_scale, mod_shift bf16
    [G, K] (or [K]), row m using row m // rows_per_group; they may be parts of
    one wider tensor and then share its row stride.  Returns
    (H, Ximg, sx, Xq, Y): the new residual stream in X's type (h_out may be X)
    and, where asked for, the bf16 image of the per-token int8 codes of y
    (image=True), their scales, the codes (codes=True) and y in bf16 (y=True);
    None otherwise."""
    if not isinstance(X, torch.Tensor) or X.dim() != 2:
        raise ValueError("X must be a [rows, width] tensor")
    if X.dtype is not torch.bfloat16 and X.dtype is not torch.float32:
        raise TypeError(f"X must be torch.bfloat16 or torch.float32, got {X.dtype}")
    m, k = X.shape
    shape, row = X.shape, (k,)
    px = _rows(X, "X", X.dtype, shape)
    pb = _rows(B, "B", torch.bfloat16, shape)
    pbg = None if branch_gamma is None else _rows(branch_gamma, "branch_gamma", torch.bfloat16, row)
    pga = None if gamma is None else _rows(gamma, "gamma", torch.bfloat16, row)
    pbe = None if beta is None else _rows(beta, "beta", torch.bfloat16, row)
    pg = ps = pt = None
    stride = 0
    if gate is not None or mod_scale is not None or mod_shift is not None:
        (pg, ps, pt), stride = _modulation((gate, mod_scale, mod_shift), k, m, rows_per_group)
    if h_out is None:
        h_out = torch.empty_like(X)
        ph = h_out.data_ptr()
    else:
        ph = _rows(h_out, "h_out", X.dtype, X.shape)
    dev = X.device
    Ximg = torch.empty((m, k), dtype=torch.bfloat16, device=dev) if image else None
    Xq = torch.empty((m, k), dtype=torch.int8, device=dev) if codes else None
    Y = torch.empty((m, k), dtype=torch.bfloat16, device=dev) if y else None
    sx = torch.empty((m,), dtype=torch.float32, device=dev) if image or codes else None
    _check("w8a8_residual_norm_quant", lib().w8a8_residual_norm_quant(
        px, pb, ph, _DTYPE[X.dtype], pbg, pga, pbe, pg, ps, pt, stride, rows_per_group, alpha, eps, kind, m, k,
        None if Y is None else Y.data_ptr(), None if Xq is None else Xq.data_ptr(),
        None if Ximg is None else Ximg.data_ptr(), None if sx is None else sx.data_ptr(),
        _raw_stream(dev.index)))
    return h_out, Ximg, sx, Xq, Y
