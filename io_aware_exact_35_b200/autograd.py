"""Autograd wrapper: exact attention as a differentiable torch operation.

``attention(q, k, v, causal, scale)`` runs the library's forward kernel and,
when gradients are needed, its recomputing backward kernel ("Flash Attention
La Gi?" (thienlv.com), Recomputation: only O and the log-sum-exp are saved,
the attention matrix is recomputed from Q, K, V).  It is a drop-in for the
scaled-dot-product attention call that "Flash Attention La Gi?" and
"DL101 chapter 9", section 3, use, restricted to what the kernels support:
bf16 q [B, H, Nq, d] and k, v [B, Hkv, Nk, d] on a B200, d in {64, 128},
Hkv dividing H (grouped-query attention).  With Nq != Nk the queries are the
last Nq positions of the key sequence, so the causal mask keeps j <= i + Nk - Nq.

``qk_norm_rope(q, k, positions, inv_freq, q_weight, k_weight)`` is the pass in
front of it: the per-head norm and the position rotation, whose backward
recomputes the norm from q and k and gives the weights' gradients too.

Both may be captured into a CUDA graph, backward included.  As with every torch
operation, no eager graph of the same leaves may be alive while a backward is
captured: torch ties the leaves' gradients to the stream of the graph that
lives, and the capture fails.
"""

from __future__ import annotations

from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from . import fa


class _Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, causal: bool, scale: Optional[float]):
        q, k, v = (t.contiguous() for t in (q, k, v))
        o, lse = fa.fwd(q, k, v, causal=causal, scale=scale)
        ctx.save_for_backward(q, k, v, o, lse)
        ctx.causal, ctx.scale = causal, scale
        return o

    @staticmethod
    def backward(ctx, do):
        q, k, v, o, lse = ctx.saved_tensors
        dq, dk, dv = fa.bwd(q, k, v, o, do.contiguous().to(torch.bfloat16), lse,
                            causal=ctx.causal, scale=ctx.scale)
        return dq, dk, dv, None, None


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, causal: bool = False,
              scale: Optional[float] = None) -> torch.Tensor:
    """softmax(scale * q k^T [+ causal mask]) v with a recomputing backward."""
    return _Attention.apply(q, k, v, bool(causal), scale)


def _rows(t: torch.Tensor) -> torch.Tensor:
    """``t``, or a copy of it in a layout the kernels read: contiguous aligned rows."""
    aligned = t.data_ptr() % 16 == 0 and all(st % 8 == 0 for st in t.stride()[:-1])
    return t if t.stride(-1) == 1 and aligned else t.clone(memory_format=torch.contiguous_format)


class _QKNormRope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, positions, inv_freq, q_weight, k_weight, eps: float,
                interleaved: bool):
        q, k = _rows(q), _rows(k)
        ctx.save_for_backward(q, k, positions, inv_freq, q_weight, k_weight)
        ctx.eps, ctx.interleaved = eps, interleaved
        return fa.qk_norm_rope(q, k, positions, inv_freq, q_weight, k_weight, eps=eps,
                               interleaved=interleaved)

    @staticmethod
    @once_differentiable  # the kernel's result has no graph: a second derivative is refused
    def backward(ctx, dq_out, dk_out):
        q, k, positions, inv_freq, q_weight, k_weight = ctx.saved_tensors
        dq, dk, dwq, dwk = fa.qk_norm_rope_bwd(q, k, _rows(dq_out), _rows(dk_out), positions,
                                               inv_freq, q_weight, k_weight, eps=ctx.eps,
                                               interleaved=ctx.interleaved)
        dwq = None if dwq is None else dwq.to(q_weight.dtype)
        dwk = None if dwk is None else dwk.to(k_weight.dtype)
        return dq, dk, None, None, dwq, dwk, None, None


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, positions: Optional[torch.Tensor],
                 inv_freq: Optional[torch.Tensor], q_weight: Optional[torch.Tensor] = None,
                 k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 interleaved: bool = False):
    """Differentiable fa.qk_norm_rope (gradients to q, k and the weights; second
    derivatives are refused)."""
    return _QKNormRope.apply(q, k, positions, inv_freq, q_weight, k_weight, float(eps),
                             bool(interleaved))
