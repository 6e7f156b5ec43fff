"""The operators between a transformer layer's W8A8 Linears.

`attention` (packed prompts, and few queries over a cache), `rotary` and
`rotary_append` (rotary positions, and the cache rows written with them) and
`residual_norm_quant` (branch norm, gate, residual, next norm, modulation and
int8 quantization in one pass).  As in the rest of the binding a function
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
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    ws = torch.empty(lib().w8a8_attention_workspace_size(), dtype=torch.uint8, device=device)
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
    of token t to row slots[t] (int64 [T]) of k_cache / v_cache [rows, Hk, D];
    a slot outside the cache (-1 for a padding token) stores nothing.  Returns
    the turned Q."""
    r = (_binding or binding()).rotary_append(Q, K, V, positions, freqs, k_cache, v_cache, slots, _layout(layout),
                                              amplitude, q_out)
    if type(r) is int:
        _check("w8a8_rotary_append", r)
    return r


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
