"""The operators between a transformer layer's W8A8 Linears.

`attention` (packed prompts, and few queries over a cache), `rotary` and
`rotary_append` (rotary positions, and the cache rows written with them),
`qk_norm_rotary` and `qk_norm_rotary_append` (the same after a norm of every query
and key head) and `residual_norm_quant` (branch norm, gate, residual, next norm,
modulation and int8 quantization in one pass); for caches in pages
`paged_attention`, `copy_pages` and `fork_sequences`.  As in the rest of the binding a function
only checks its tensors, allocates outputs and passes pointers, sizes and the
current stream to the library (include/w8a8.h states the arithmetic); here that
is done in C++ (csrc/binding.cpp), as it would take longer than the kernels of
single tokens.  Nothing synchronizes, so every call can be captured into a CUDA
graph.  Nothing is recorded for a backward pass; a tensor that is written in
place (an output given, a cache) must not require a gradient outside
torch.no_grad(), and autograd knows it as changed.
"""
import importlib.machinery
import importlib.util
import math
import os

import torch

from . import LIB_PATH, RMS_NORM, _check, lib

HALF = "half"
INTERLEAVED = "interleaved"

_LAYOUT = {HALF: 0, INTERLEAVED: 1}

_binding = None


def binding():
    """Load csrc/binding.cpp's module (raises if it has not been built)."""
    global _binding
    if _binding is None:
        path = os.path.join(os.path.dirname(LIB_PATH), f"w8a8_binding_torch{torch.__version__}.so")
        if not os.path.exists(path):
            raise RuntimeError(f"W8A8 binding not built ({path} missing): run __graft_entry__.build()")
        lib()
        loader = importlib.machinery.ExtensionFileLoader("w8a8_binding", path)
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("w8a8_binding", loader))
        loader.exec_module(module)
        _binding = module
    return _binding


def attention_workspace(device=None):
    """A workspace for `attention`, for one stream at a time (the counters at
    its start are, and stay between calls, zero)."""
    return _workspace(lib().w8a8_attention_workspace_size(), device)


def _workspace(size, device):
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    ws = torch.empty(size, dtype=torch.uint8, device=device)
    ws[:lib().w8a8_attention_workspace_zeroed()].zero_()
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

    Returns O [Tq, Hq, D], or (O, lse fp32 [Tq, Hq]) with lse=True.  `out`
    must not overlap Q, K or V.  The workspace (`attention_workspace()`, 10 MB)
    is by default one per stream, kept until the process ends, and one of its
    own, in the graph's memory, for a captured call."""
    r = (_binding or binding()).attention(Q, K, V, cu_q, cu_k, k_lens, batch, causal, scale, out, lse, workspace)
    if type(r) is int:
        _check("w8a8_attention", r)
    return r


def rotary_frequencies(rot_dim, base=10000.0, scaling=None, factor=1.0, original_length=None, fast=32.0, slow=1.0,
                       device="cuda", ramp="turns"):
    """Radians per position of each of the rot_dim / 2 pairs, fp64 [rot_dim / 2]:
    base ** (-2 k / rot_dim), for a context `factor` times longer than trained:
      "linear": all divided by factor;
      "ntk":    base * factor ** (rot_dim / (rot_dim - 2)), which divides the
                slowest pair's frequency by factor and leaves the fastest;
      "yarn":   (Peng et al. 2023) pairs that turn more than `fast` times in
                original_length positions are kept, those below `slow` turns
                divided by factor, with a ramp in between; used with the
                amplitude rotary_amplitude(factor) = 0.1 ln(factor) + 1.
    "yarn" has two ramps, and a trained model needs its own (frequencies in between
    differ by factors of up to 4).  ramp="turns" is the paper's formula, linear in
    the number of turns; ramp="pairs" is linear in the pair's index, from the index
    that has `fast` turns, rounded down, to the one that has `slow`, rounded up, as
    in the authors' code and the models that follow it."""
    if rot_dim <= 0 or rot_dim % 2:
        raise ValueError("rot_dim must be even and positive")
    if scaling not in (None, "linear", "ntk", "yarn"):
        raise ValueError("scaling must be None, 'linear', 'ntk' or 'yarn'")
    if ramp not in ("turns", "pairs"):
        raise ValueError("ramp must be 'turns' or 'pairs'")
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
        if original_length is None or not fast > slow or (ramp == "pairs" and not slow > 0):
            raise ValueError("'yarn' needs original_length, and fast > slow (above 0 with ramp='pairs')")
        if ramp == "turns":
            keep = ((original_length * f / (2 * math.pi) - slow) / (fast - slow)).clamp(0, 1)
        else:
            # original_length * base ** (-2 k / rot_dim) = 2 pi turns, solved for k
            first, last = (rot_dim / 2 * math.log(original_length / (2 * math.pi * turns)) / math.log(base)
                           for turns in (fast, slow))
            first, last = max(math.floor(first), 0), min(math.ceil(last), rot_dim - 1)
            pair = torch.arange(rot_dim // 2, dtype=torch.float64)
            keep = 1 - ((pair - first) / max(last - first, 1e-3)).clamp(0, 1)
        f = f * keep + f / factor * (1 - keep)
    return f.to(device)


def rotary_amplitude(factor):
    """The amplitude that goes with "yarn" frequencies."""
    return 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0


def _layout(layout):
    if layout not in _LAYOUT:
        raise ValueError("layout must be 'half' or 'interleaved'")
    return _LAYOUT[layout]


def rotary(Q, K, positions, freqs, layout=HALF, amplitude=1.0, inverse=False, q_out=None, k_out=None):
    """Rotary positions of Q [T, Hq, D] and K [T, Hk, D] (or None): the first
    2 * len(freqs) elements of each head turn by positions[t] * freqs[k]
    (int64 [T], fp64 from `rotary_frequencies`), the rest is copied.  Returns
    (Q', K'), new tensors unless q_out / k_out are given; these may be Q and K
    themselves.  inverse=True turns back (also the gradient's direction, at
    amplitude 1)."""
    r = (_binding or binding()).rotary(Q, K, positions, freqs, _layout(layout), amplitude, inverse, q_out, k_out)
    if type(r) is int:
        _check("w8a8_rotary", r)
    return r


def rotary_append(Q, K, V, positions, freqs, k_cache, v_cache, slots, layout=HALF, amplitude=1.0, q_out=None):
    """`rotary` for tokens that join a cache: turns Q and K, and writes K and V
    of token t to row slots[t] (int64 [T]) of k_cache / v_cache: rows
    [rows, Hk, D], or pages [pages, page_size, Hk, D], where row
    page * page_size + i is row i of a page (any strides, the last dimension
    dense).  A slot outside the cache (-1 for a padding token) stores nothing.
    Returns the turned Q."""
    r = (_binding or binding()).rotary_append(Q, K, V, positions, freqs, k_cache, v_cache, slots, _layout(layout),
                                              amplitude, q_out)
    if type(r) is int:
        _check("w8a8_rotary_append", r)
    return r


def qk_norm_rotary(Q, K, positions, freqs, q_gamma=None, k_gamma=None, eps=1e-6, kind=RMS_NORM, layout=HALF,
                   amplitude=1.0, q_out=None, k_out=None):
    """`rotary` of Q [T, Hq, D] and K [T, Hk, D] (or None) after a norm of every
    head: RMSNorm (or LayerNorm without shift, kind=LAYER_NORM) over its D
    elements, times q_gamma / k_gamma ([D], or [heads, D], of Q's type; None: 1),
    in binary32 up to one rounding of the result.  Returns (Q', K'), new tensors
    unless q_out / k_out are given; these may be Q and K themselves."""
    r = (_binding or binding()).qk_norm_rotary(Q, K, positions, freqs, q_gamma, k_gamma, eps, kind, _layout(layout),
                                               amplitude, q_out, k_out)
    if type(r) is int:
        _check("w8a8_qk_norm_rotary", r)
    return r


def qk_norm_rotary_append(Q, K, V, positions, freqs, k_cache, v_cache, slots, q_gamma=None, k_gamma=None, eps=1e-6,
                          kind=RMS_NORM, layout=HALF, amplitude=1.0, q_out=None):
    """`qk_norm_rotary` for tokens that join a cache: K, normed and turned, and V
    of token t go to row slots[t] (int64 [T]) of k_cache / v_cache, rows or pages
    as in `rotary_append`.  A slot outside the cache (-1 for a padding token) stores
    nothing.  Returns the normed and turned Q."""
    r = (_binding or binding()).qk_norm_rotary_append(Q, K, V, positions, freqs, k_cache, v_cache, slots, q_gamma,
                                                      k_gamma, eps, kind, _layout(layout), amplitude, q_out)
    if type(r) is int:
        _check("w8a8_qk_norm_rotary_append", r)
    return r


def paged_attention_workspace(device=None):
    """A workspace for `paged_attention`, for one stream at a time."""
    return _workspace(lib().w8a8_paged_attention_workspace_size(), device)


def paged_attention(Q, k_pages, v_pages, page_table, k_lens, cu_q=None, max_queries=None, causal=True, scale=None,
                    out=None, lse=False, workspace=None):
    """`attention` of new tokens over a cache in pages: from one to thousands of
    them for each sequence, of both kinds in one call.

    Q [Tq, Hq, D] as in `attention`; k_pages, v_pages [pages, page_size, Hk, D]
    (any strides, the last dimension dense; page_size a multiple of 8).  Key j of
    sequence b is row j % page_size of page page_table[b, j // page_size]
    (int32 [B, most pages]; what lies past the last page is not read, an entry
    outside the cache reads as zeros).  k_lens: int32 [B] keys of each sequence,
    its new tokens (which are in the cache already) included.  cu_q: int32
    [B + 1] first rows of the sequences' queries; without it the rows are B equal
    parts.  max_queries: the most queries of a sequence, where the host knows it; it
    only chooses between kernels (which may round differently).  A batch of single
    tokens passes max_queries=1 with its cu_q, or no cu_q where every sequence has a
    token; otherwise it is served like a chunk in a batch with idle sequences, which
    looks the same to the host (unless every sequence has a row and Tq * Hq / Hk <= 64).
    causal, scale, out and lse as in `attention`; rows of no sequence are not written.

    The workspace (`paged_attention_workspace()`, 51 MB) is by default one per
    stream, kept until the process ends, and one of its own, in the graph's
    memory, for a captured call."""
    r = (_binding or binding()).paged_attention(Q, k_pages, v_pages, page_table, k_lens, cu_q, max_queries, causal,
                                                scale, out, lse, workspace)
    if type(r) is int:
        _check("w8a8_paged_attention", r)
    return r


def copy_pages(caches, src, dst):
    """Page dst[i] = page src[i] (int32 [n], on the GPU) in every one of `caches`:
    a list of tensors [pages, ...] with dense pages, such as every layer's k_pages
    and v_pages.  A pair with an index outside the cache (-1) copies nothing.  No
    page may be a destination twice, or a destination and a source.

    A cache is compacted by copies of its last pages to free ones before them, and
    map[page_table] with map = arange(pages), map[src] = dst."""
    r = (_binding or binding()).copy_pages(caches, src, dst)
    if type(r) is int:
        _check("w8a8_copy_pages", r)


def fork_sequences(caches, page_table, k_lens, src, dst, new_pages, page_size):
    """Sequence dst[i] (a row of page_table [rows, most pages] and of k_lens
    [rows], int32) becomes a second one like src[i] that can go on by itself: it
    gets its length and its full pages, and page new_pages[i] for what comes next,
    into which the last page is copied, in every one of `caches` (as in
    `copy_pages`), where it is only partly filled.  src, dst, new_pages: int32 [n],
    on the GPU.  Nothing happens where src[i] == dst[i], or where a row or the
    new page is outside the table or the cache (-1).  A row may be the source of
    many, but no row a destination twice, or a destination and a source, and no
    new page used twice or part of a sequence.  Which pages are free, and how many
    sequences share one, is the caller's to know."""
    r = (_binding or binding()).fork_sequences(caches, page_table, k_lens, src, dst, new_pages, page_size)
    if type(r) is int:
        _check("w8a8_fork_sequences", r)


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
    r = (_binding or binding()).residual_norm_quant(X, B, gamma, beta, eps, kind, alpha, gate, branch_gamma, mod_scale,
                                                    mod_shift, rows_per_group, h_out, image, codes, y)
    if type(r) is int:
        _check("w8a8_residual_norm_quant", r)
    return r
