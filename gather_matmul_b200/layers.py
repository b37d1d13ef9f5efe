"""The attention inputs of one decoder layer whose q/k/v projection carries
LoRA adapters: the library's calls in the order a serving step makes them.

  y        = x W^T                                   linear_fp8
  y       += scale (x A[idx]^T) B[idx]^T  per slice  bgmv
  y[q, k]  = rotation of (the norms of) the heads    norm_rope / rope, in place

All work is enqueued on the current stream; no call allocates, so a step can
be captured in a CUDA graph.
"""
from typing import Optional, Sequence

import torch

from . import ops


class AttentionInputs:
    """One layer's weights and the workspaces of batches of up to max_tokens
    tokens.

    W, w_scale   float8_e4m3fn [N, K] and its block scales (quantize_fp8 with
                 block_rows=128); the N columns of y are the q heads, the k
                 heads, then the v heads.
    A, B         LoRA stacks of the q, k and v slices, as for ops.bgmv (A may be
                 one shared stack), contiguous and of x's dtype.
    inv_freq, attn_scale   from ops.rope_frequencies.
    q_norm, k_norm         [head_dim] weights of the head norms; both None for a
                           layer without them.

    Calls of one object share its workspaces: calls that may overlap on the
    GPU (two streams, two captured graphs replayed at once) need an object
    each.
    """

    def __init__(self, W: torch.Tensor, w_scale: torch.Tensor, A: Sequence[torch.Tensor],
                 B: Sequence[torch.Tensor], q_heads: int, kv_heads: int, head_dim: int,
                 inv_freq: torch.Tensor, max_tokens: int, scale: float = 1.0,
                 attn_scale: float = 1.0, interleaved: bool = False,
                 q_norm: Optional[torch.Tensor] = None, k_norm: Optional[torch.Tensor] = None,
                 eps: float = 1e-6):
        widths = [q_heads * head_dim, kv_heads * head_dim, kv_heads * head_dim]
        if W.shape[0] != sum(widths) or [b.shape[1] for b in B] != widths:
            raise ValueError("W's rows and B's stacks must be the q, k and v heads")
        S, r, K = A[0].shape
        if K != W.shape[1] or any(a.shape != A[0].shape for a in A) or \
                any(b.shape[0] != S or b.shape[2] != r for b in B):
            raise ValueError("A must be [S, r, K] stacks for W's K columns, B [S, width, r]")
        if len(A) not in (1, len(B)):
            raise ValueError("A must hold one stack per slice, or one shared stack")
        # the kernels take the stacks by address alone
        if any(t.dtype is not A[0].dtype for t in (*A, *B)):
            raise TypeError("A and B must be of one dtype, that of x")
        if not all(t.is_contiguous() and t.device == W.device for t in (*A, *B)):
            raise ValueError("A and B must be contiguous and on W's device")
        self.W, self.w_scale, self.A, self.B = W, w_scale, list(A), list(B)
        self.heads, self.head_dim = [q_heads, kv_heads], head_dim
        self.inv_freq, self.attn_scale, self.interleaved = inv_freq, attn_scale, interleaved
        self.norms = None if q_norm is None and k_norm is None else [q_norm, k_norm]
        self.eps, self.scale, self.max_tokens = eps, scale, max_tokens
        self.work = ops.linear_fp8_workspace(max_tokens, K, W.device)
        self.meta = ops.workspace(max_tokens, S, W.device)
        self.buf = torch.empty(len(A) * max_tokens * r, dtype=torch.float32, device=W.device)

    def __call__(self, x: torch.Tensor, idx: torch.Tensor, positions: torch.Tensor,
                 y: torch.Tensor, has_lora: Optional[bool] = None, idx_host=None) -> torch.Tensor:
        """y [T, N] (overwritten) from x [T, K], adapter indices and positions.
        has_lora / idx_host as has_active / idx_host of ops.bgmv."""
        T = x.shape[0]
        if T > self.max_tokens:
            raise ValueError(f"{T} tokens; the workspaces hold {self.max_tokens}")
        if x.dtype is not self.A[0].dtype:
            raise TypeError(f"x must be {self.A[0].dtype}, as the LoRA stacks are")
        if idx.device != self.W.device:
            raise ValueError("idx must be on W's device")
        ops.linear_fp8(x, self.W, self.w_scale, y, self.work)
        r = self.A[0].shape[1]
        buf = self.buf[:len(self.A) * T * r].view(len(self.A), T, r)
        ops.bgmv(x, self.A, self.B, idx, y, buf, self.meta, self.scale, has_active=has_lora,
                 idx_host=idx_host)
        if self.norms is None:
            return ops.rope(y, y, self.heads, self.head_dim, positions, self.inv_freq,
                            interleaved=self.interleaved, attn_scale=self.attn_scale)
        return ops.norm_rope(y, self.norms, y, self.heads, self.head_dim, positions, self.inv_freq,
                             eps=self.eps, interleaved=self.interleaved,
                             attn_scale=self.attn_scale)
