"""Linear attention with a decay for each head, over whole sequences.

    S_t = e^g S_{t-1} + k_t v_t^T,    o_t = scale S_t^T q_t

taken by the chunk, forward and backward; the shapes, the grouped value heads, the packed sequences and the states are
those of ``chunk_gated_delta_rule``, so that both kinds of layers share a model's layout and a pool of states.
``recurrent_linear_attention`` goes on from the final states token by token.

    q, k [B,T,Hq,K], v [B,T,Hv,V]  bf16 or fp32, K and V 64 or 128, Hv a multiple of Hq; any strides whose last
                                   dimension is contiguous
    g [Hv]                         the logarithm of each head's decay, 0 or below (None: no decay).  It is a constant of
                                   the layer, as in retention: it has no gradient, and one that is asked for is refused
    initial_state [N,Hv,K,V]       fp32, N = B or the number of packed sequences
    cu_seqlens [N+1]               B = 1: the sequences' offsets, read on the GPU alone.  A sequence whose offsets fall or leave the
                                   T tokens counts as empty; rows outside every sequence are 0 in all outputs

A NaN or an infinity in a token reaches the outputs of its sequence's chunk of 64 tokens and of what comes behind it, and no
other sequence.  The gradients of k, v and the initial state run from the last token to the first: there it reaches the chunk,
counted from the sequence's end, and what comes before it.

The calls go through the extension module (``csrc/binding.cpp``), synchronise nothing and read nothing back, so that they can be
captured in a CUDA graph.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import decode as _decode

__all__ = ["chunk_linear_attention", "chunk_linear_attention_fwd", "chunk_linear_attention_bwd"]


def _native():
    return _decode._native or _decode.load_binding()


def chunk_linear_attention_fwd(q, k, v, g=None, scale=None, initial_state=None, output_final_state=True, cu_seqlens=None):
    """(o, final_state); final_state is None unless wanted."""
    return _native().linear_fwd(q, k, v, g, scale, initial_state, cu_seqlens, output_final_state)


def chunk_linear_attention_bwd(q, k, v, g, do, dht=None, scale=None, initial_state=None, cu_seqlens=None):
    """(dq, dk, dv, dh0) from the gradients of o and, where there is one, of the final state; dh0 is None without an
    initial state."""
    return _native().linear_bwd(q, k, v, g, scale, initial_state, cu_seqlens, do, dht, 7 if initial_state is None else 15)


class _LinearAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, scale, initial_state, output_final_state, cu_seqlens):
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(q, k, v, g, initial_state, cu_seqlens)
        ctx.scale = scale
        return _native().linear_fwd(q, k, v, g, scale, initial_state, cu_seqlens, output_final_state)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, do, dht):
        q, k, v, g, h0, cu = ctx.saved_tensors
        needs = ctx.needs_input_grad
        if do is None and dht is None:
            return (None,) * 8
        if do is None:
            do = torch.zeros_like(v)
        wanted = needs[0] | needs[1] << 1 | needs[2] << 2 | (h0 is not None and needs[5]) << 3
        dq, dk, dv, dh0 = _native().linear_bwd(q, k, v, g, ctx.scale, h0, cu, do, dht, wanted)
        return dq, dk, dv, None, None, dh0, None, None


def chunk_linear_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: Optional[torch.Tensor] = None,
                           scale: Optional[float] = None, initial_state: Optional[torch.Tensor] = None,
                           output_final_state: bool = False, cu_seqlens: Optional[torch.Tensor] = None):
    """Returns (o, final_state); final_state is None unless asked for.  q, k, v and initial_state have gradients."""
    if torch.is_grad_enabled():
        if g is not None and g.requires_grad:
            raise ValueError("g is a constant of the layer and has no gradient: detach it")
        if q.requires_grad or k.requires_grad or v.requires_grad or (initial_state is not None and initial_state.requires_grad):
            return _LinearAttention.apply(q, k, v, g, scale, initial_state, bool(output_final_state), cu_seqlens)
    return _native().linear_fwd(q, k, v, g, scale, initial_state, cu_seqlens, output_final_state)
