"""Decoding with the gated delta rule: the calls that follow a prefill.

``chunk_gated_delta_rule(..., output_final_state=True)`` leaves one state per sequence; kept in a pool
``[slots, Hv, K, V]`` (fp32), it is moved on and read by

    o = recurrent_gated_delta_rule(q, k, v, g, beta, state, state_indices=...)   # new tokens, in place
    o = tree_gated_delta_rule(q, k, v, g, beta, parents, state, ...)             # drafted tokens, state kept
    scores, tokens, parents = beam_search_step(logits, scores, ...)              # one selection
    reorder_states(states, parents, ...)                                         # the states follow it

Marshalling onto the decoding entry points of ``include/gdn.h``, which also says what happens to indices that
are out of range.  Nothing here synchronises or copies to the host, so the calls can be captured in a CUDA
graph.  There is no CPU path and no backward: training runs through ``chunk_gated_delta_rule``.
"""
from __future__ import annotations

import ctypes
import struct
from typing import Optional, Sequence, Union

import torch
from torch._C import _cuda_getCurrentRawStream as _raw_stream

from . import GDN_BF16, GDN_F32, GdnError, load_library

__all__ = ["recurrent_gated_delta_rule", "tree_gated_delta_rule", "beam_search_step", "reorder_states",
           "TREE_MAX", "BEAM_MAX"]

TREE_MAX = 64
BEAM_MAX = 64
_CODES = {torch.bfloat16: GDN_BF16, torch.float32: GDN_F32}
_I64 = ctypes.c_int64
_P = ctypes.c_void_p

# A decoding call takes a few microseconds on the GPU, so its way there is kept short: the C structures are packed
# in one go (a ctypes structure of this size takes longer to fill than a launch) and the stream is taken as a number.
#   gdn_decode_problem: B T Hq Hv K V, (batch, token, head) strides of q k v g beta, io_dtype scale, n_slots
#   slot_stride, state_indices, n_seqs, cu_seqlens, token_indices, n_steps
_DECODE = struct.Struct("@6q15qif2qPqPPq")
#   gdn_beam_problem: B W vocab n, strides of logits and mask, dtype
_BEAM = struct.Struct("@8qi0q")
#   gdn_state_view
_VIEW = struct.Struct("@P2q")

_lib = None


def _library():
    global _lib
    if _lib is None:
        lib = load_library()
        C = ctypes.c_char_p
        lib.gdn_recurrent.argtypes = [C] + [_P] * 9
        lib.gdn_tree.argtypes = [C] + [_P] * 9
        lib.gdn_beam_search_workspace_bytes.argtypes = [C]
        lib.gdn_beam_search_workspace_bytes.restype = ctypes.c_size_t
        lib.gdn_beam_search.argtypes = [C] + [_P] * 8 + [ctypes.c_size_t, _P]
        lib.gdn_reorder_states.argtypes = [C] + [_I64] * 4 + [_P] * 3
        for f in (lib.gdn_recurrent, lib.gdn_tree, lib.gdn_beam_search, lib.gdn_reorder_states):
            f.restype = ctypes.c_int
        _lib = lib
    return _lib


def _device(t: torch.Tensor, name: str) -> torch.device:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path)")
    return t.device


def _shape(t: torch.Tensor, name: str, shape, device):
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")


def _ints(t: Optional[torch.Tensor], name: str, shape, device) -> Optional[torch.Tensor]:
    """Device indices as contiguous int32."""
    if t is None:
        return None
    _shape(t, name, shape, device)
    if t.dtype != torch.int32:
        if t.dtype not in (torch.int64, torch.int16, torch.int8, torch.uint8):
            raise TypeError(f"{name} must hold integers, got {t.dtype}")
        t = t.to(torch.int32)
    return t.contiguous()


def _ptr(t: Optional[torch.Tensor]):
    return 0 if t is None else t.data_ptr()


def _call(where: str, fn, device: torch.device, *args):
    index = device.index
    if index != torch.cuda.current_device():
        with torch.cuda.device(device):
            rc = fn(*args, _raw_stream(index))
    else:
        rc = fn(*args, _raw_stream(index))
    if rc != 0:
        raise GdnError(rc, where)


def _inputs(q, k, v, g, beta, state):
    """Checks what the two state operators share and makes the layouts that the kernels read."""
    dev = _device(k, "k")
    if k.dim() != 4 or v.dim() != 4:
        raise ValueError("k and v must have four dimensions: [B, T, heads, width]")
    B, T, _, K = k.shape
    Hv, V = v.shape[2:]
    dtype = k.dtype
    if dtype not in _CODES:
        raise TypeError(f"unsupported io dtype {dtype} (bfloat16 or float32)")
    grad = k.requires_grad or v.requires_grad or g.requires_grad or beta.requires_grad or state.requires_grad
    if q is not None:
        _shape(q, "q", k.shape, dev)
        if q.dtype != dtype:
            raise TypeError("q, k and v must have one dtype")
        grad = grad or q.requires_grad
        if q.stride(3) != 1:
            q = q.contiguous()
    _shape(v, "v", (B, T, Hv, V), dev)
    _shape(g, "g", (B, T, Hv), dev)
    _shape(beta, "beta", (B, T, Hv), dev)
    if v.dtype != dtype:
        raise TypeError("q, k and v must have one dtype")
    if grad and torch.is_grad_enabled():
        raise ValueError("the decoding operators have no backward: call them under torch.no_grad(), or train through "
                         "chunk_gated_delta_rule")
    if state.dim() != 4 or state.shape[1:] != (Hv, K, V):
        raise ValueError(f"state must have shape (slots, {Hv}, {K}, {V}), got {tuple(state.shape)}")
    if state.dtype != torch.float32:
        raise TypeError(f"state must be float32, got {state.dtype}")
    if state.device != dev:
        raise ValueError(f"state must be on {dev}, got {state.device}")
    if not state.is_contiguous() and state.stride()[1:] != (K * V, V, 1):
        raise ValueError("every slot of state must be contiguous")
    if k.stride(3) != 1:
        k = k.contiguous()
    if v.stride(3) != 1:
        v = v.contiguous()
    if g.dtype != torch.float32:
        g = g.float()
    if beta.dtype != torch.float32:
        beta = beta.float()
    return dev, q, k, v, g, beta


def _problem(q, k, v, g, beta, state, scale, state_indices, n_seqs, cu_seqlens=None, token_indices=None, n_steps=0):
    B, T, Hq, K = k.shape
    Hv, V = v.shape[2:]
    k0, k1, k2, _ = k.stride()
    q0, q1, q2, _ = k.stride() if q is None else q.stride()
    v0, v1, v2, _ = v.stride()
    return _DECODE.pack(B, T, Hq, Hv, K, V, q0, q1, q2, k0, k1, k2, v0, v1, v2, *g.stride(), *beta.stride(),
                        _CODES[k.dtype], K ** -0.5 if scale is None else scale, state.shape[0], state.stride(0),
                        _ptr(state_indices), n_seqs, _ptr(cu_seqlens), _ptr(token_indices), n_steps)


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
    cu_seqlens [N+1]   B = 1: N sequences packed one after the other, one slot each.
    token_indices [B,P]  run row n through its tokens token_indices[n, 0], [n, 1], ... up to the first negative
                       entry: the accepted path of a drafted tree, or rows of different lengths.  o is [B,P,Hv,V].
    out_state [B,Hv,K,V]  (or [N,...]) gets the new states, row by row, and ``state`` is only read: rows may then
                       share a slot, as beams that continue one parent do.  Must not overlap ``state``.
    q = None           only the states move; returns None.
    """
    dev, q, k, v, g, beta = _inputs(q, k, v, g, beta, state)
    B, steps, Hv, V = v.shape
    n_seqs = B
    if cu_seqlens is not None:
        if B != 1:
            raise ValueError("cu_seqlens needs B = 1")
        if token_indices is not None:
            raise ValueError("token_indices and cu_seqlens exclude each other")
        if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
            raise ValueError("cu_seqlens must have one dimension and at least one entry")
        cu_seqlens = _ints(cu_seqlens, "cu_seqlens", cu_seqlens.shape, dev)
        n_seqs = cu_seqlens.shape[0] - 1
    if token_indices is not None:
        if token_indices.dim() != 2:
            raise ValueError("token_indices must have two dimensions")
        steps = token_indices.shape[1]
        token_indices = _ints(token_indices, "token_indices", (B, steps), dev)
    state_indices = _ints(state_indices, "state_indices", (n_seqs,), dev)
    if out_state is not None:
        _shape(out_state, "out_state", (n_seqs,) + state.shape[1:], dev)
        if out_state.dtype != torch.float32 or not out_state.is_contiguous():
            raise ValueError("out_state must be contiguous float32")
    p = _problem(q, k, v, g, beta, state, scale, state_indices, n_seqs, cu_seqlens, token_indices,
                 0 if token_indices is None else steps)
    o = None if q is None else torch.empty((B, steps, Hv, V), dtype=k.dtype, device=dev)
    _call("gdn_recurrent", _library().gdn_recurrent, dev, p, _ptr(q), k.data_ptr(), v.data_ptr(), g.data_ptr(),
          beta.data_ptr(), state.data_ptr(), _ptr(out_state), _ptr(o))
    return o


def tree_gated_delta_rule(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
                          parents: torch.Tensor, state: torch.Tensor, scale: Optional[float] = None,
                          state_indices: Optional[torch.Tensor] = None) -> torch.Tensor:
    """A tree of drafted tokens per sequence, answered from its state, which stays as it is.

    parents [B,T]: for each token the earlier token of its row that it follows, -1 if it follows the state
    itself; below -1 the token is absent (o = 0), and with it what follows it.  At most TREE_MAX tokens.  Other
    arguments as recurrent_gated_delta_rule.  Returns o [B,T,Hv,V]: what each token's path would give.  Move the
    state along the accepted path with recurrent_gated_delta_rule(None, ..., token_indices=path).
    """
    if q is None:
        raise ValueError("q must be given")
    dev, q, k, v, g, beta = _inputs(q, k, v, g, beta, state)
    B = k.shape[0]
    state_indices = _ints(state_indices, "state_indices", (B,), dev)
    parents = _ints(parents, "parents", k.shape[:2], dev)
    p = _problem(q, k, v, g, beta, state, scale, state_indices, B)
    o = torch.empty(v.shape, dtype=k.dtype, device=dev)
    _call("gdn_tree", _library().gdn_tree, dev, p, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(),
          beta.data_ptr(), parents.data_ptr(), state.data_ptr(), o.data_ptr())
    return o


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
    dev = _device(logits, "logits")
    if logits.dim() != 3:
        raise ValueError("logits must have three dimensions: [B, W, vocab]")
    B, W, vocab = logits.shape
    if logits.dtype not in _CODES:
        raise TypeError(f"unsupported logits dtype {logits.dtype} (bfloat16 or float32)")
    n = W if num_candidates is None else int(num_candidates)
    if not 1 <= n <= BEAM_MAX or not 1 <= W <= BEAM_MAX:
        raise ValueError(f"beams and candidates must be 1 to {BEAM_MAX}")
    _shape(scores, "scores", (B, W), dev)
    if scores.dtype != torch.float32:
        raise TypeError(f"scores must be float32, got {scores.dtype}")
    if logits.stride(2) != 1:
        logits = logits.contiguous()
    scores = scores.contiguous()
    mask_batch = mask_beam = 0
    if finished is not None:
        _shape(finished, "finished", (B, W), dev)
        if finished.dtype != torch.bool:
            raise TypeError(f"finished must be bool, got {finished.dtype}")
        finished = finished.contiguous()
    if mask is not None:
        if mask.dtype != torch.bool:
            raise TypeError(f"mask must be bool, got {mask.dtype}")
        if mask.device != dev:
            raise ValueError(f"mask must be on {dev}, got {mask.device}")
        if mask.shape != logits.shape:
            try:
                mask = mask.expand(B, W, vocab)
            except RuntimeError:
                raise ValueError(f"mask must be broadcastable to {(B, W, vocab)}, got {tuple(mask.shape)}") from None
        if mask.stride(2) != 1:
            mask = mask.contiguous()
        mask_batch, mask_beam, _ = mask.stride()
    lib = _library()
    p = _BEAM.pack(B, W, vocab, n, logits.stride(0), logits.stride(1), mask_batch, mask_beam, _CODES[logits.dtype])
    need = lib.gdn_beam_search_workspace_bytes(p)
    if need == 0:
        raise GdnError(2, "gdn_beam_search")
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    out_scores = torch.empty((B, n), dtype=torch.float32, device=dev)
    tokens = torch.empty((B, n), dtype=torch.int32, device=dev)
    parents = torch.empty((B, n), dtype=torch.int32, device=dev)
    _call("gdn_beam_search", lib.gdn_beam_search, dev, p, logits.data_ptr(), scores.data_ptr(), _ptr(finished),
          _ptr(mask), out_scores.data_ptr(), tokens.data_ptr(), parents.data_ptr(), workspace.data_ptr(),
          workspace.numel() * workspace.element_size())
    return out_scores, tokens, parents


def reorder_states(states: Union[torch.Tensor, Sequence[torch.Tensor]], parents: torch.Tensor,
                   state_indices: Optional[torch.Tensor] = None) -> None:
    """The states of every beam become those of its parent, in place, for all tensors at once.

    states: one tensor or several, each [slots, ...] of any dtype with contiguous slots (the layers' states, the
    last inputs of their short convolutions, ...).  parents [B,W]: beam i of search b continues beam
    parents[b,i] of the same search; negative: it stays as it is.  state_indices [B,W]: the beams' slots, which
    must differ (default: b * W + i); negative: an idle beam.
    """
    if isinstance(states, torch.Tensor):
        states = (states,)
    if not states:
        return
    dev = _device(states[0], "states")
    if parents.dim() != 2:
        raise ValueError("parents must have two dimensions: [B, W]")
    B, W = parents.shape
    if not 1 <= W <= BEAM_MAX:
        raise ValueError(f"beams must be 1 to {BEAM_MAX}")
    parents = _ints(parents, "parents", (B, W), dev)
    state_indices = _ints(state_indices, "state_indices", (B, W), dev)
    slots = states[0].shape[0]
    views = b""
    for s in states:
        if s.dim() < 1 or s.shape[0] != slots:
            raise ValueError("all states must have the same number of slots")
        if s.device != dev:
            raise ValueError(f"states must be on {dev}, got {s.device}")
        if not s.is_contiguous() and s.numel() and not s[0].is_contiguous():
            raise ValueError("every slot of a state must be contiguous")
        size = s.element_size()
        views += _VIEW.pack(s.data_ptr(), s.stride(0) * size, s.numel() // slots * size if slots else 0)
    _call("gdn_reorder_states", _library().gdn_reorder_states, dev, views, len(states), slots, B, W,
          parents.data_ptr(), _ptr(state_indices))
