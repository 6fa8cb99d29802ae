"""A decoder layer around the sparse FFN, from the library's calls: a serving step for the new tokens of up to
DECODE_MAX_N sequences, and the training step of the FFN's half of the layer.

The residual stream travels as (delta, h): what the last sublayer added and the stream before it. The
addition itself is the first half of twell_add_rmsnorm_fwd, so a sublayer reads and writes the stream once.
Positions are the caller's business: `rotate`, if given, is called with the queries and keys of a step (views of
the fused projection's output, to be changed in place) before the keys are stored.
With a `stream`, a step runs under it: its kernels, what `rotate` queues, and the memory of what it returns.
"""
from __future__ import annotations

import dataclasses
from typing import Callable, Optional

import torch

from . import binding


@dataclasses.dataclass
class DecoderLayer:
    """Weights of one layer: norms in bf16, 4-bit projections (binding.twell_w4_quantize), the FFN's Wg_s, Wu_s and
    Wd_s. w_qkv has n_heads query rows blocks, then n_kv_heads key and n_kv_heads value ones, of head_dim rows each."""

    attn_norm: torch.Tensor  # [d]
    w_qkv: binding.W4Weights  # [(n_heads + 2 n_kv_heads) head_dim, d]
    w_out: binding.W4Weights  # [d, n_heads head_dim]
    ffn_norm: torch.Tensor  # [d]
    Wg_s: torch.Tensor
    Wu_s: torch.Tensor
    Wd_s: torch.Tensor
    n_heads: int
    n_kv_heads: int
    head_dim: int
    eps: float = 1e-6
    T: int = 128
    rotate: Optional[Callable[[torch.Tensor, torch.Tensor], None]] = None

    def decode(self, delta: torch.Tensor, h: Optional[torch.Tensor], cache: binding.KVCache, slots: torch.Tensor,
               page_table: torch.Tensor, seq_lens: torch.Tensor, window: int = 0, stream=None):
        """One new token per sequence: delta [N, d] bf16 and h [N, d] (bf16 or fp32; None for the first layer, whose
        stream is delta) in, the same pair for the next layer out. The tokens' keys and values go to
        `slots`; seq_lens counts them."""
        N = delta.shape[0]
        hq, hk = self.n_heads, self.n_kv_heads
        with binding.under_stream(stream):
            y, h1, _ = binding.twell_add_rmsnorm_fwd(delta, self.attn_norm, h, self.eps)
            h1 = delta if h1 is None else h1
            qkv = binding.twell_w4_matvec(y, self.w_qkv).view(N, hq + 2 * hk, self.head_dim)
            q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
            if self.rotate is not None:
                self.rotate(q, k)
            binding.twell_kv_append(cache, k, v, slots)
            a, _ = binding.twell_paged_attn_decode(q, cache, page_table, seq_lens, window=window)
            o = binding.twell_w4_matvec(a.view(N, hq * self.head_dim), self.w_out)
            y, h2, _ = binding.twell_add_rmsnorm_fwd(o, self.ffn_norm, h1, self.eps)
            return binding.ffn_forward(y, self.Wg_s, self.Wu_s, self.Wd_s, T=self.T, path="auto"), h2


def ffn_sublayer_fwd(delta, h, ffn_norm, Wg_s, Wu_s, Wd_s, K: int, backup_cap: int, l1_coef: float = 2e-5,
                     eps: float = 1e-6, stream=None):
    """The FFN's half of a layer, training: h' = delta + h (h None: delta), f = FFN(norm(h')). Returns (f, h', saved)."""
    with binding.under_stream(stream):
        y, h1, rstd = binding.twell_add_rmsnorm_fwd(delta, ffn_norm, h, eps, training=True)
        h1 = delta if h1 is None else h1
        f, ctx = binding.twell_hybrid_fwd(y, Wg_s, Wu_s, Wd_s, K, backup_cap, l1_coef)
    return f, h1, (y, h1, rstd, ctx, ffn_norm, Wg_s, Wu_s, Wd_s, l1_coef)


def ffn_sublayer_bwd(df, dh, saved, stream=None):
    """Gradients of <f, df> + <h', dh> + the L1 term: df bf16, dh fp32 (the gradient that reaches h' from the
    layers above). Returns (d, dffn_norm, dWg_s, dWu_s, dWd_s), all fp32; d is the gradient of delta and h alike."""
    y, h1, rstd, ctx, ffn_norm, Wg_s, Wu_s, Wd_s, l1_coef = saved
    with binding.under_stream(stream):
        dy, dWg, dWu, dWd = binding.twell_hybrid_bwd(y, Wg_s, Wu_s, Wd_s, ctx, df, l1_coef)
        d, dn = binding.twell_add_rmsnorm_bwd(dy, h1, ffn_norm, rstd, dh, dx=dy)
    return d, dn, dWg, dWu, dWd
