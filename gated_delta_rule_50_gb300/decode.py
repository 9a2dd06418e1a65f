"""Decoding with the gated delta rule and with linear attention: the calls that follow a prefill.

``chunk_gated_delta_rule(..., output_final_state=True)`` leaves one state per sequence; kept in a pool
``[slots, Hv, K, V]`` (fp32), it is moved on and read by

    o = recurrent_gated_delta_rule(q, k, v, g, beta, state, state_indices=...)   # new tokens, in place
    o = tree_gated_delta_rule(q, k, v, g, beta, parents, state, ...)             # drafted tokens, state kept
    scores, tokens, parents = beam_search_step(logits, scores, ...)              # one selection
    reorder_states(states, parents, ...)                                         # the states follow it
    tokens, logprobs = sample_tokens(logits, random, ...)                        # or one token drawn per row

``recurrent_linear_attention`` is the step for states that ``chunk_linear_attention`` left.

The calls go through an extension module (``csrc/binding.cpp``) onto the decoding entry points of
``include/gdn.h``, which also says what happens to indices that are out of range (whatever integers hold them: they
are read as int32, and what does not fit stays out of range).  Nothing here synchronises or copies to the host, so
the calls can be captured in a CUDA graph.  There is no CPU path and no derivative: training runs through
``chunk_gated_delta_rule`` and ``chunk_linear_attention``, and inputs that require a gradient or carry a tangent are refused (under
``torch.no_grad()`` the former are taken).
"""
from __future__ import annotations

import importlib.machinery
import importlib.util
import threading
from typing import Optional, Sequence, Union

import torch

from . import GdnError, load_library
from . import build as _build

__all__ = ["recurrent_gated_delta_rule", "tree_gated_delta_rule", "beam_search_step", "reorder_states",
           "recurrent_linear_attention", "sample_tokens", "load_binding", "TREE_MAX", "BEAM_MAX"]

TREE_MAX = 64
BEAM_MAX = 64

_native = None
_lock = threading.Lock()


def load_binding():
    """Builds (if needed) and loads the extension module; raises if either fails."""
    global _native
    with _lock:
        if _native is None:
            path = _build.build_binding()
            load_library()
            loader = importlib.machinery.ExtensionFileLoader("_gdn_decode", path)
            module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_gdn_decode", loader))
            loader.exec_module(module)
            module.set_errors(GdnError, torch.OutOfMemoryError)
            _native = module
    return _native


def recurrent_gated_delta_rule(q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                               beta: torch.Tensor, state: torch.Tensor, scale: Optional[float] = None,
                               state_indices: Optional[torch.Tensor] = None,
                               cu_seqlens: Optional[torch.Tensor] = None,
                               token_indices: Optional[torch.Tensor] = None,
                               out_state: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
    """New tokens of every sequence, one after the other; ``state`` is updated in place.

    q, k [B,T,Hq,K]; v [B,T,Hv,V] (bf16 or fp32, any strides with a contiguous last dimension); g, beta
    [B,T,Hv]; state [slots,Hv,K,V] fp32.  Returns o [B,T,Hv,V].

    state_indices [B]  the slot of each row (default: row n has slot n); negative: an idle row, o = 0.  The
                       slots of one call must differ unless ``out_state`` is given.
    cu_seqlens [N+1]   B = 1: N sequences packed one after the other, one slot each.  Tokens outside every sequence
                       have o = 0; so have those of a sequence whose offsets fall or leave the T tokens, unless
                       another claims them, and its slot stays as it was.
    token_indices [B,P]  run row n through its tokens token_indices[n, 0], [n, 1], ... up to the first negative
                       entry: the accepted path of a drafted tree, or rows of different lengths.  o is [B,P,Hv,V].
    out_state [B,Hv,K,V]  (or [N,...]) gets the new states, row by row, and ``state`` is only read: rows may then
                       share a slot, as beams that continue one parent do.  Must not overlap ``state``.
    q = None           only the states move; returns None.
    """
    return (_native or load_binding()).recurrent(q, k, v, g, beta, state, scale, state_indices, cu_seqlens, token_indices,
                                                 out_state)


def recurrent_linear_attention(q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor, g: Optional[torch.Tensor],
                               state: torch.Tensor, scale: Optional[float] = None,
                               state_indices: Optional[torch.Tensor] = None,
                               cu_seqlens: Optional[torch.Tensor] = None,
                               token_indices: Optional[torch.Tensor] = None,
                               out_state: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
    """New tokens of every sequence through linear attention, S <- e^g S + k v^T and o = scale S^T q; ``state`` is
    updated in place.

    g [Hv]: the logarithm of each head's decay (None: no decay).  Everything else as in recurrent_gated_delta_rule.
    """
    return (_native or load_binding()).linear_recurrent(q, k, v, g, None, state, scale, state_indices, cu_seqlens,
                                                        token_indices, out_state)


def tree_gated_delta_rule(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
                          parents: torch.Tensor, state: torch.Tensor, scale: Optional[float] = None,
                          state_indices: Optional[torch.Tensor] = None) -> torch.Tensor:
    """A tree of drafted tokens per sequence, answered from its state, which stays as it is.

    parents [B,T]: for each token the earlier token of its row that it follows, -1 if it follows the state
    itself; below -1 the token is absent (o = 0), and with it what follows it.  At most TREE_MAX tokens.  Other
    arguments as recurrent_gated_delta_rule.  Returns o [B,T,Hv,V]: what each token's path would give.  Move the
    state along the accepted path with recurrent_gated_delta_rule(None, ..., token_indices=path).
    """
    return (_native or load_binding()).tree(q, k, v, g, beta, state, scale, state_indices, parents)


def beam_search_step(logits: torch.Tensor, scores: torch.Tensor, finished: Optional[torch.Tensor] = None,
                     mask: Optional[torch.Tensor] = None, num_candidates: Optional[int] = None,
                     workspace: Optional[torch.Tensor] = None):
    """The best continuations of each search, best first: (scores fp32, tokens int32, parents int32), [B,n] each.

    logits [B,W,vocab] (bf16 or fp32, the vocabulary contiguous); scores [B,W] the beams' sums of log
    probabilities so far (-inf: no such beam); finished [B,W] bool: such a beam competes as it is, its token is
    -1; mask bool, broadcastable to logits: False forbids a token, whatever its logit holds.  n = num_candidates
    (default W).  A candidate's score is its beam's plus the log-softmax of the allowed logits; equal ones go by
    the lower beam, then the lower token.  Where fewer than n candidates are left: score -inf, token -1, parent
    j % W.
    """
    return (_native or load_binding()).beam(logits, scores, finished, mask, num_candidates, workspace)


def sample_tokens(logits: torch.Tensor, random: torch.Tensor, temperature: Union[float, torch.Tensor] = 1.0,
                  top_k: Union[int, torch.Tensor, None] = None, top_p: Union[float, torch.Tensor, None] = None,
                  min_p: Union[float, torch.Tensor, None] = None, mask: Optional[torch.Tensor] = None):
    """One token for each row, drawn with a given random number: (tokens int32 [B], logprobs fp32 [B]).

    logits [B,vocab] (bf16 or fp32, the vocabulary contiguous, B and vocab up to 2^20); random [B] fp32 in [0, 1);
    temperature, top_k, top_p and min_p are numbers or tensors [B], one for each row; mask bool, broadcastable to logits:
    False forbids a token, whatever its logit holds.

    Of the allowed tokens, best first and equal ones by the lower token, the ``top_k`` first are kept (0 or below: all);
    of these, with shares softmax(logits / temperature), the fewest whose shares sum to ``top_p`` at least (1 or above:
    all); of these those with ``min_p`` times the best one's share at least.  What is left is run through in the order
    of the vocabulary: the token is the first where the running sum of shares exceeds ``random`` times their sum, its
    logprob the logarithm of its part in that sum.  temperature 0: the best token, logprob 0.  A row without a choice
    (nothing allowed, a NaN or +inf among what is, a parameter that is none) has the token -1 and the logprob -inf.
    """
    return (_native or load_binding()).sample(logits, random, temperature, top_k, top_p, min_p, mask)


def reorder_states(states: Union[torch.Tensor, Sequence[torch.Tensor]], parents: torch.Tensor,
                   state_indices: Optional[torch.Tensor] = None) -> None:
    """The states of every beam become those of its parent, in place, for all tensors at once.

    states: one tensor or several, each [slots, ...] of any dtype with contiguous slots (the layers' states, the
    last inputs of their short convolutions, ...).  parents [B,W]: beam i of search b continues beam
    parents[b,i] of the same search; negative: it stays as it is.  state_indices [B,W]: the beams' slots, which
    must differ (default: b * W + i); negative: an idle beam.
    """
    (_native or load_binding()).reorder(states, parents, state_indices)
