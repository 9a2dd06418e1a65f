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
from typing import Optional, Sequence, Union

import torch

from . import GDN_BF16, GDN_F32, GdnError, load_library

__all__ = ["recurrent_gated_delta_rule", "tree_gated_delta_rule", "beam_search_step", "reorder_states",
           "TREE_MAX", "BEAM_MAX"]

TREE_MAX = 64
BEAM_MAX = 64
_CODES = {torch.bfloat16: GDN_BF16, torch.float32: GDN_F32}
_I64 = ctypes.c_int64
_P = ctypes.c_void_p


class _Strides(ctypes.Structure):
    _fields_ = [("batch", _I64), ("token", _I64), ("head", _I64)]


class _DecodeProblem(ctypes.Structure):
    _fields_ = ([(n, _I64) for n in ("B", "T", "Hq", "Hv", "K", "V")]
                + [(n, _Strides) for n in ("q", "k", "v", "g", "beta")]
                + [("io_dtype", ctypes.c_int), ("scale", ctypes.c_float), ("n_slots", _I64), ("slot_stride", _I64),
                   ("state_indices", _P), ("n_seqs", _I64), ("cu_seqlens", _P), ("token_indices", _P),
                   ("n_steps", _I64)])


class _BeamProblem(ctypes.Structure):
    _fields_ = ([(n, _I64) for n in ("B", "W", "vocab", "n", "logits_batch", "logits_beam", "mask_batch", "mask_beam")]
                + [("logits_dtype", ctypes.c_int)])


class _StateView(ctypes.Structure):
    _fields_ = [("data", _P), ("slot_stride", _I64), ("slot_bytes", _I64)]


_lib = None


def _library():
    global _lib
    if _lib is None:
        lib = load_library()
        dp, bp = ctypes.POINTER(_DecodeProblem), ctypes.POINTER(_BeamProblem)
        lib.gdn_recurrent.argtypes = [dp] + [_P] * 9
        lib.gdn_tree.argtypes = [dp] + [_P] * 9
        lib.gdn_beam_search_workspace_bytes.argtypes = [bp]
        lib.gdn_beam_search_workspace_bytes.restype = ctypes.c_size_t
        lib.gdn_beam_search.argtypes = [bp] + [_P] * 8 + [ctypes.c_size_t, _P]
        lib.gdn_reorder_states.argtypes = [ctypes.POINTER(_StateView)] + [_I64] * 4 + [_P] * 3
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
    return None if t is None else t.data_ptr()


def _call(where: str, fn, device: torch.device, *args):
    if device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            rc = fn(*args, torch.cuda.current_stream(device).cuda_stream)
    else:
        rc = fn(*args, torch.cuda.current_stream(device).cuda_stream)
    if rc != 0:
        raise GdnError(rc, where)


def _problem(q, k, v, g, beta, state, scale, state_indices):
    """Checks what the two state operators share; returns (problem, tensors that it points to)."""
    dev = _device(k, "k")
    if k.dim() != 4 or v.dim() != 4:
        raise ValueError("k and v must have four dimensions: [B, T, heads, width]")
    B, T, Hq, K = k.shape
    Hv, V = v.shape[2], v.shape[3]
    if k.dtype not in _CODES:
        raise TypeError(f"unsupported io dtype {k.dtype} (bfloat16 or float32)")
    if q is not None:
        _shape(q, "q", k.shape, dev)
    _shape(v, "v", (B, T, Hv, V), dev)
    for t, name in ((g, "g"), (beta, "beta")):
        _shape(t, name, (B, T, Hv), dev)
    if v.dtype != k.dtype or (q is not None and q.dtype != k.dtype):
        raise TypeError("q, k and v must have one dtype")
    if torch.is_grad_enabled() and (k.requires_grad or v.requires_grad or g.requires_grad or beta.requires_grad
                                    or state.requires_grad or (q is not None and q.requires_grad)):
        raise ValueError("the decoding operators have no backward: call them under torch.no_grad(), or train through "
                         "chunk_gated_delta_rule")
    if state.dim() != 4 or state.shape[1:] != (Hv, K, V):
        raise ValueError(f"state must have shape (slots, {Hv}, {K}, {V}), got {tuple(state.shape)}")
    if state.dtype != torch.float32:
        raise TypeError(f"state must be float32, got {state.dtype}")
    if state.device != dev:
        raise ValueError(f"state must be on {dev}, got {state.device}")
    if state.numel() and state.stride()[1:] != (K * V, V, 1):
        raise ValueError("every slot of state must be contiguous")
    if k.stride(3) != 1:
        k = k.contiguous()
    if v.stride(3) != 1:
        v = v.contiguous()
    if q is not None and q.stride(3) != 1:
        q = q.contiguous()
    if g.dtype != torch.float32:
        g = g.float()
    if beta.dtype != torch.float32:
        beta = beta.float()
    p = _DecodeProblem()
    p.B, p.T, p.Hq, p.Hv, p.K, p.V = B, T, Hq, Hv, K, V
    if q is not None:
        p.q = q.stride()[:3]
    p.k, p.v, p.g, p.beta = k.stride()[:3], v.stride()[:3], g.stride(), beta.stride()
    p.io_dtype = _CODES[k.dtype]
    p.scale = K ** -0.5 if scale is None else scale
    p.n_slots, p.slot_stride = state.shape[0], state.stride(0)
    p.state_indices = _ptr(state_indices)
    return p, q, k, v, g, beta


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
    dev = _device(k, "k")
    n_seqs = k.shape[0]
    if cu_seqlens is not None:
        if k.shape[0] != 1:
            raise ValueError("cu_seqlens needs B = 1")
        if token_indices is not None:
            raise ValueError("token_indices and cu_seqlens exclude each other")
        if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
            raise ValueError("cu_seqlens must have one dimension and at least one entry")
        cu_seqlens = _ints(cu_seqlens, "cu_seqlens", cu_seqlens.shape, dev)
        n_seqs = cu_seqlens.shape[0] - 1
    state_indices = _ints(state_indices, "state_indices", (n_seqs,), dev)
    p, q, k, v, g, beta = _problem(q, k, v, g, beta, state, scale, state_indices)
    B, T, Hv, V = v.shape
    p.n_seqs, p.cu_seqlens = n_seqs, _ptr(cu_seqlens)
    steps = T
    if token_indices is not None:
        if token_indices.dim() != 2:
            raise ValueError("token_indices must have two dimensions")
        steps = token_indices.shape[1]
        token_indices = _ints(token_indices, "token_indices", (B, steps), dev)
        p.token_indices, p.n_steps = _ptr(token_indices), steps
    if out_state is not None:
        _shape(out_state, "out_state", (n_seqs,) + state.shape[1:], dev)
        if out_state.dtype != torch.float32 or not out_state.is_contiguous():
            raise ValueError("out_state must be contiguous float32")
    o = None if q is None else torch.empty(B, steps, Hv, V, dtype=k.dtype, device=dev)
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
    dev = _device(k, "k")
    if q is None:
        raise ValueError("q must be given")
    state_indices = _ints(state_indices, "state_indices", (k.shape[0],), dev)
    parents = _ints(parents, "parents", k.shape[:2], dev)
    p, q, k, v, g, beta = _problem(q, k, v, g, beta, state, scale, state_indices)
    p.n_seqs = k.shape[0]
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
    p = _BeamProblem(B, W, vocab, n, logits.stride(0), logits.stride(1), 0, 0, _CODES[logits.dtype])
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
        try:
            mask = mask.expand(B, W, vocab)
        except RuntimeError:
            raise ValueError(f"mask must be broadcastable to {(B, W, vocab)}, got {tuple(mask.shape)}") from None
        if mask.stride(2) != 1:
            mask = mask.contiguous()
        p.mask_batch, p.mask_beam = mask.stride(0), mask.stride(1)
    lib = _library()
    need = lib.gdn_beam_search_workspace_bytes(p)
    if need == 0:
        raise GdnError(2, "gdn_beam_search")
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    out_scores = torch.empty(B, n, dtype=torch.float32, device=dev)
    tokens = torch.empty(2, B, n, dtype=torch.int32, device=dev)
    parents = tokens[1]
    tokens = tokens[0]
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
    views = (_StateView * len(states))()
    for view, s in zip(views, states):
        if s.dim() < 1 or s.shape[0] != slots:
            raise ValueError("all states must have the same number of slots")
        if s.device != dev:
            raise ValueError(f"states must be on {dev}, got {s.device}")
        if s.numel() and not s[0].is_contiguous():
            raise ValueError("every slot of a state must be contiguous")
        size = s.element_size()
        view.data, view.slot_stride = s.data_ptr(), s.stride(0) * size
        view.slot_bytes = s.numel() // slots * size if slots else 0
    _call("gdn_reorder_states", _library().gdn_reorder_states, dev, views, len(states), slots, B, W,
          parents.data_ptr(), _ptr(state_indices))
