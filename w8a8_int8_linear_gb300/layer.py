"""Int8TransformerLayer: a decoder layer whose Linears are W8A8 and whose other
operators are this package's, for whole prompts and for single tokens.

    qkv = Linear(RMSNorm(x))             norm and quantization in one pass
    q, k = rotary(q, k); k, v -> cache   one kernel
    a = attention(q, cache)
    h, u = x + Linear(a), RMSNorm(h)     residual and norm in one pass
    y = h + FFN(u)

"TurboDiffusion Integration Notes", section "Reused Components", names the
pieces around the W8A8 Linear: fused norms, modulation / residual / rotary
helpers and attention.
"""
import torch

from .module import Int8FFN, Int8Linear
from .operators import HALF, attention, residual_norm_quant, rotary_append


class Int8TransformerLayer(torch.nn.Module):
    """x [T, width] bf16 -> y [T, width], T the new tokens of all sequences one
    after another.  qkv_weight [(heads + 2 * kv_heads) * dim, width], out_weight
    [width, heads * dim], up_weight [hidden, width], down_weight
    [width, hidden]; attn_norm / ffn_norm [width]; frequencies from
    `rotary_frequencies`."""

    def __init__(self, qkv_weight, out_weight, up_weight, down_weight, heads, kv_heads, attn_norm, ffn_norm,
                 frequencies, layout=HALF, amplitude=1.0, eps=1e-6):
        super().__init__()
        rows = qkv_weight.shape[0]
        if rows % (heads + 2 * kv_heads) or heads % kv_heads:
            raise ValueError("qkv_weight must have (heads + 2 * kv_heads) * dim rows, heads a multiple of kv_heads")
        self.heads, self.kv_heads, self.dim = heads, kv_heads, rows // (heads + 2 * kv_heads)
        self.qkv = Int8Linear(qkv_weight, norm="rms", norm_weight=attn_norm, eps=eps)
        self.out = Int8Linear(out_weight)
        self.ffn = Int8FFN(up_weight, down_weight)
        self.register_buffer("ffn_norm", ffn_norm.detach().to(torch.bfloat16).contiguous())
        self.register_buffer("frequencies", frequencies)
        self.layout, self.amplitude, self.eps = layout, amplitude, eps

    def new_cache(self, batch, capacity):
        """K and V for `batch` sequences of up to `capacity` tokens."""
        shape = (batch * capacity, self.kv_heads, self.dim)
        return tuple(torch.zeros(shape, dtype=torch.bfloat16, device=self.ffn_norm.device) for _ in range(2))

    def forward(self, x, positions, k_cache, v_cache, slots, k_lens, batch, cu_q=None):
        """positions, slots: int64 [T], each token's position and its row of the
        caches [batch * capacity, kv_heads, dim]; k_lens: int32 [batch] tokens
        in each sequence's part of the cache, the new ones included; cu_q:
        int32 [batch + 1] the sequences' first rows of x (None: equally many
        tokens of each).  Each token sees its sequence's tokens up to itself."""
        t = x.shape[0]
        qkv = self.qkv(x).view(t, self.heads + 2 * self.kv_heads, self.dim)
        q, k, v = qkv.split((self.heads, self.kv_heads, self.kv_heads), dim=1)
        q = rotary_append(q, k, v, positions, self.frequencies, k_cache, v_cache, slots, self.layout, self.amplitude)
        a = attention(q, k_cache, v_cache, cu_q=cu_q, k_lens=k_lens, batch=batch)
        h, _, _, _, u = residual_norm_quant(x, self.out(a.view(t, -1)), gamma=self.ffn_norm, eps=self.eps,
                                            image=False, y=True)
        return h + self.ffn(u)

    def extra_repr(self):
        return f"heads={self.heads}, kv_heads={self.kv_heads}, dim={self.dim}"
