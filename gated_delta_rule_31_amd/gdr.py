"""The gated delta rule with one decay per value head, and decoding with drafted tokens.

* ``gdr_chunk_fwd(q, k, v, g, beta, ...)`` -- prefill: g and beta per value head, q and k
  shared by the HV / HK value heads of a group; packed sequences, initial and final states.
* ``gdr_chunk_bwd(q, k, v, g, beta, d_out, ...)`` -- its gradients; ``gated_delta_rule(q, k, v,
  g, beta, ...)`` -- the prefill recorded for autograd through them.
* ``gdr_recurrent_step(q, k, v, g, beta, states, ...)`` -- decode: one or several tokens a
  request over a pool of states, the state after every drafted token in a slot of its own;
  a decay per value head, or per channel as KDA has it.
* ``draft_verify(target_probs, draft_tokens, uniforms, ...)`` -- which drafted tokens hold
  against the target's probabilities, and the token behind them; its ``accepted`` is the
  next ``gdr_recurrent_step``'s ``start``.
"""
from __future__ import annotations

import functools
from typing import Optional, Tuple

import torch

from . import _check, _dtype_code, _forward, _load, _needs_grad, _no_tangent


def _input(x: Optional[torch.Tensor], name: str, like: Optional[torch.Tensor] = None, dtype=None, border: int = 16) -> Optional[torch.Tensor]:
    """A dense tensor on the device of ``like``, on a border of ``border`` bytes (copied to one if need be):
    16 for what the kernels read in wide loads, 4 for what they read number by number."""
    if x is None:
        return None
    if not isinstance(x, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if _forward._current_level >= 0:
        _no_tangent(x, name)
    if like is None:
        if not x.is_cuda:
            raise ValueError("%s must be on the GPU (got %s)" % (name, x.device))
    elif x.device != like.device:
        raise ValueError("%s is on %s, but the first input is on %s" % (name, x.device, like.device))
    if dtype is not None and x.dtype != dtype:
        raise ValueError("%s must be %s (got %s)" % (name, dtype, x.dtype))
    if x.requires_grad and torch.is_grad_enabled():
        raise ValueError("%s requires grad: the raw kernels do not record autograd; use the recorded call (gated_delta_rule, short_conv, gated_linear_recurrence, block_norm), or the call for its gradients yourself" % name)
    if not x.is_contiguous():
        x = x.contiguous()
    return x.clone() if x.data_ptr() % border else x


def _p(x: Optional[torch.Tensor]):
    return None if x is None else x.data_ptr()


# the current stream's handle without a Stream object around it (2 us of a 14 us call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)


def _call(fn, device: torch.device, *args) -> None:
    """A C entry point on the device's current stream; the device is made current where it is not."""
    if torch.cuda.current_device() == device.index:
        st = fn(*args, _raw_stream(device.index))
    else:
        with torch.cuda.device(device):
            st = fn(*args, _raw_stream(device.index))
    if st:
        _check(fn.__name__, st)


def _output(x: torch.Tensor, name: str, shape, dtype, device) -> torch.Tensor:
    """A caller's buffer that is written in place: it has to be what the kernels write as it is."""
    if (not isinstance(x, torch.Tensor) or tuple(x.shape) != tuple(shape) or x.dtype != dtype or x.device != device
            or not x.is_contiguous()):
        raise ValueError("%s must be a contiguous %s tensor %s on %s" % (name, dtype, list(shape), device))
    if _forward._current_level >= 0:
        _no_tangent(x, name)
    if x.requires_grad and torch.is_grad_enabled():
        raise ValueError("%s requires grad: it is written in place" % name)
    return x


def _workspace(x: Optional[torch.Tensor], need: int, device) -> torch.Tensor:
    if x is None:
        return torch.empty(max(need, 1), dtype=torch.uint8, device=device)
    if x.device != device or x.dtype != torch.uint8 or not x.is_contiguous() or x.numel() < need:
        raise ValueError("workspace must be a contiguous uint8 tensor of at least %d bytes on %s" % (need, device))
    return x


def _chunk_inputs(q, k, v, g, beta, initial_state, cu_seqlens):
    q = _input(q, "q")
    if q is None:
        raise TypeError("q must be a torch.Tensor")
    k, v = _input(k, "k", q, q.dtype), _input(v, "v", q, q.dtype)
    g, beta = _input(g, "g", q, torch.float32, 4), _input(beta, "beta", q, torch.float32, 4)
    initial_state = _input(initial_state, "initial_state", q, torch.float32)
    cu_seqlens = _input(cu_seqlens, "cu_seqlens", q, torch.int32, 4)
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k must be [B, T, HK, K] and v [B, T, HV, V]")
    B, T, HK, K = q.shape
    HV, V = v.shape[2:]
    if k.shape != q.shape or v.shape[:2] != (B, T) or g.shape != (B, T, HV) or beta.shape != (B, T, HV):
        raise ValueError("inconsistent shapes: q %s k %s v %s g %s beta %s" % tuple(tuple(x.shape) for x in (q, k, v, g, beta)))
    if cu_seqlens is not None and (cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1):
        raise ValueError("cu_seqlens must be int32 [N + 1]")
    N = B if cu_seqlens is None else cu_seqlens.numel() - 1
    if initial_state is not None and initial_state.shape != (N, HV, K, V):
        raise ValueError("initial_state must be %s" % [N, HV, K, V])
    return q, k, v, g, beta, initial_state, cu_seqlens, (B, T, HK, HV, K, V, N)


@functools.lru_cache(maxsize=256)
def _workspace_size(fn: str, *shape: int) -> int:
    """A workspace's size by its shape alone."""
    return int(getattr(_load(), fn)(*shape))


def gdr_chunk_fwd_workspace_size(dtype: torch.dtype, B: int, T: int, HK: int, HV: int, K: int, V: int, num_seqs: int = 0,
                                 varlen: bool = False) -> int:
    """Bytes of device workspace ``gdr_chunk_fwd`` needs for this shape (0: unsupported or empty)."""
    return _workspace_size("kda_gdr_chunk_fwd_workspace_size", _dtype_code(dtype), int(B), int(T), int(num_seqs), 1 if varlen else 0, int(HK),
                           int(HV), int(K), int(V))


def gdr_chunk_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
                  initial_state: Optional[torch.Tensor] = None, output_final_state: bool = True,
                  cu_seqlens: Optional[torch.Tensor] = None, scale: float = 1.0, out_dtype: Optional[torch.dtype] = None,
                  out: Optional[torch.Tensor] = None, final_state: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Prefill of the gated delta rule.  q, k [B,T,HK,K]; v [B,T,HV,V] (one dtype, float32 or
    bfloat16; HV a multiple of HK); g [B,T,HV] float32 log decays (<= 0, -inf allowed); beta
    [B,T,HV] float32; initial_state [N,HV,K,V] float32 or None (zeros); cu_seqlens int32 [N+1]
    (B == 1) or None.  Returns (out [B,T,HV,V], final_state [N,HV,K,V] or None).  ``final_state``
    may be passed in (it may be ``initial_state``).  Rows of ``out`` behind the last packed
    sequence are left as they were (unset in an ``out`` made here)."""
    q, k, v, g, beta, initial_state, cu_seqlens, (B, T, HK, HV, K, V, N) = _chunk_inputs(q, k, v, g, beta, initial_state, cu_seqlens)
    od, dev = out_dtype or v.dtype, q.device
    if out is None:
        out = torch.empty((B, T, HV, V), dtype=od, device=dev)
    else:
        out = _output(out, "out", (B, T, HV, V), od, dev)
    if final_state is None:
        final_state = torch.empty((N, HV, K, V), dtype=torch.float32, device=dev) if output_final_state else None
    else:
        final_state = _output(final_state, "final_state", (N, HV, K, V), torch.float32, dev)
    workspace = _workspace(workspace, gdr_chunk_fwd_workspace_size(q.dtype, B, T, HK, HV, K, V, N, cu_seqlens is not None), dev)
    _call(_load().kda_gdr_chunk_fwd, dev, _p(q), _p(k), _p(v), _dtype_code(q.dtype), _p(g), _p(beta), _p(initial_state), _p(final_state),
          _p(cu_seqlens), N, B, T, HK, HV, K, V, float(scale), _p(out), _dtype_code(od), _p(workspace), workspace.numel())
    return out, final_state


def gdr_chunk_bwd_workspace_size(dtype: torch.dtype, B: int, T: int, HK: int, HV: int, K: int, V: int, num_seqs: int = 0,
                                 varlen: bool = False) -> int:
    """Bytes of device workspace ``gdr_chunk_bwd`` needs for this shape (0: unsupported or empty)."""
    return _workspace_size("kda_gdr_chunk_bwd_workspace_size", _dtype_code(dtype), int(B), int(T), int(num_seqs), 1 if varlen else 0, int(HK),
                           int(HV), int(K), int(V))


def gdr_chunk_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor, d_out: torch.Tensor,
                  initial_state: Optional[torch.Tensor] = None, d_final_state: Optional[torch.Tensor] = None,
                  cu_seqlens: Optional[torch.Tensor] = None, scale: float = 1.0, grad_dtype: Optional[torch.dtype] = None,
                  want_d_initial_state: bool = True, workspace: Optional[torch.Tensor] = None):
    """Gradients of ``gdr_chunk_fwd`` (same q, k, v, g, beta, initial_state, cu_seqlens, scale) for
    L = <d_out, out> + <d_final_state, final_state>.  Returns (dq, dk, dv, dg, dbeta,
    d_initial_state): dq, dk (summed over the value heads of a group) and dv in ``grad_dtype``
    (default: the dtype of q), dg and dbeta [B,T,HV] float32, d_initial_state [N,HV,K,V] float32
    or None.  Rows behind the last packed sequence get zeros.  ``workspace``: a uint8 CUDA tensor
    of at least ``gdr_chunk_bwd_workspace_size`` bytes, allocated here if not given."""
    q, k, v, g, beta, initial_state, cu_seqlens, (B, T, HK, HV, K, V, N) = _chunk_inputs(q, k, v, g, beta, initial_state, cu_seqlens)
    d_out, d_final_state = _input(d_out, "d_out", q), _input(d_final_state, "d_final_state", q, torch.float32)
    if d_out is None or d_out.shape != v.shape:
        raise ValueError("d_out must be shaped like v")
    if d_final_state is not None and d_final_state.shape != (N, HV, K, V):
        raise ValueError("d_final_state must be %s" % [N, HV, K, V])
    gd, dev = grad_dtype or q.dtype, q.device
    dq, dk, dv = (torch.empty(x.shape, dtype=gd, device=dev) for x in (q, k, v))
    dg, dbeta = (torch.empty(g.shape, dtype=torch.float32, device=dev) for _ in range(2))
    ds0 = torch.empty((N, HV, K, V), dtype=torch.float32, device=dev) if want_d_initial_state else None
    workspace = _workspace(workspace, gdr_chunk_bwd_workspace_size(q.dtype, B, T, HK, HV, K, V, N, cu_seqlens is not None), dev)
    _call(_load().kda_gdr_chunk_bwd, dev, _p(q), _p(k), _p(v), _dtype_code(q.dtype), _p(g), _p(beta), _p(initial_state), _p(cu_seqlens), N, B,
          T, HK, HV, K, V, float(scale), _p(d_out), _dtype_code(d_out.dtype), _p(d_final_state), _p(dq), _p(dk), _p(dv), _dtype_code(gd), _p(dg),
          _p(dbeta), _p(ds0), _p(workspace), workspace.numel())
    return dq, dk, dv, dg, dbeta, ds0


def _zeros_behind(q, k, v, g, beta, initial_state, cu_seqlens, scale):
    """``gdr_chunk_fwd`` with zeros behind the last packed sequence."""
    out = None if cu_seqlens is None else torch.zeros_like(v, memory_format=torch.contiguous_format)
    return gdr_chunk_fwd(q, k, v, g, beta, initial_state=initial_state, cu_seqlens=cu_seqlens, scale=scale, out=out)


class _GatedDeltaRuleFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, beta, initial_state, cu_seqlens, scale):
        d = lambda x: None if x is None else x.detach()  # noqa: E731
        with torch.no_grad():
            out, fin = _zeros_behind(d(q), d(k), d(v), d(g), d(beta), d(initial_state), cu_seqlens, scale)
        ctx.save_for_backward(q, k, v, g, beta, initial_state, cu_seqlens)
        ctx.scale = scale
        ctx.set_materialize_grads(False)
        return out, fin

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, d_out, d_fin):
        q, k, v, g, beta, s0, cu = ctx.saved_tensors
        if d_out is None:
            d_out = torch.zeros(v.shape, dtype=v.dtype, device=v.device)
        d = lambda x: None if x is None else x.detach()  # noqa: E731
        with torch.no_grad():
            dq, dk, dv, dg, db, ds0 = gdr_chunk_bwd(d(q), d(k), d(v), d(g), d(beta), d_out, initial_state=d(s0), d_final_state=d_fin,
                                                    cu_seqlens=cu, scale=ctx.scale, want_d_initial_state=ctx.needs_input_grad[5])
        return dq, dk, dv, dg, db, ds0, None, None


def gated_delta_rule(q, k, v, g, beta, initial_state=None, cu_seqlens=None, scale: float = 1.0):
    """``gdr_chunk_fwd`` as a function of its inputs: (out in the inputs' dtype, final_state), recorded
    for autograd when any of q, k, v, g, beta or initial_state requires grad (through
    ``gdr_chunk_bwd``).  Rows of out behind the last packed sequence are zeros, whether the call is
    recorded or not."""
    if _needs_grad(q, k, v, g, beta, initial_state):
        return _GatedDeltaRuleFn.apply(q, k, v, g, beta, initial_state, cu_seqlens, float(scale))
    return _zeros_behind(q, k, v, g, beta, initial_state, cu_seqlens, scale)


def gdr_recurrent_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor, states: torch.Tensor,
                       slots: Optional[torch.Tensor] = None, start: Optional[torch.Tensor] = None,
                       lengths: Optional[torch.Tensor] = None, scale: float = 1.0, out_dtype: Optional[torch.dtype] = None,
                       out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Up to S tokens for each of B requests over a pool of states.  q, k [B,S,HK,K]; v
    [B,S,HV,V]; g [B,S,HV] float32 log decays, or [B,S,HV,K], one per channel; beta [B,S,HV]
    float32; states [pool,HV,K,V] float32 contiguous, updated in place.

    slots int32 [B, S]: the state after each token goes to a slot of its own (a slot outside the
    pool keeps none), and a request starts from ``slots[b, start[b]]``, ``start`` int32 [B] being
    the number of drafts that held in the round before (None: column 0); rounds that follow one
    another keep one table and one S, and give fewer tokens by ``lengths``.  slots [B] or [B, 1]: a request starts from
    its slot and leaves the state after its last token there; None: slot b.  A slot that one
    request writes must not be named by another.  lengths int32 [B]: tokens of each request
    (None: S); rows of ``out`` behind them are left as they were (zeros in an ``out`` made here).
    Returns out [B,S,HV,V]."""
    q = _input(q, "q")
    if q is None:
        raise TypeError("q must be a torch.Tensor")
    k, v = _input(k, "k", q, q.dtype), _input(v, "v", q, q.dtype)
    g, beta = _input(g, "g", q, torch.float32, 4), _input(beta, "beta", q, torch.float32, 4)
    if g.dim() == 4:  # decays per channel are read in wide loads
        g = _input(g, "g", q, torch.float32)
    slots, start, lengths = (_input(x, n, q, torch.int32, 4) for x, n in ((slots, "slots"), (start, "start"), (lengths, "lengths")))
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k must be [B, S, HK, K] and v [B, S, HV, V]")
    B, S, HK, K = q.shape
    HV, V = v.shape[2:]
    if k.shape != q.shape or v.shape[:2] != (B, S) or beta.shape != (B, S, HV) or tuple(g.shape) not in ((B, S, HV), (B, S, HV, K)):
        raise ValueError("inconsistent shapes: q %s k %s v %s g %s beta %s" % tuple(tuple(x.shape) for x in (q, k, v, g, beta)))
    dev = q.device
    if not isinstance(states, torch.Tensor) or states.dim() != 4:
        raise ValueError("states must be [pool, HV, K, V]")
    pool = states.shape[0]
    states = _output(states, "states", (pool, HV, K, V), torch.float32, dev)
    cols = 1
    if slots is not None:
        cols = 1 if slots.dim() == 1 else slots.shape[-1]
        if slots.dim() not in (1, 2) or slots.shape[0] != B or cols not in (1, S):
            raise ValueError("slots must be [B], [B, 1] or [B, S]")
    if slots is None and (start is not None or pool < B):
        raise ValueError("without slots every request has a state of its own, states[b], and starts from it")
    if start is not None and cols != S:
        raise ValueError("start names a column of slots [B, S]")
    if (start is not None and start.shape != (B,)) or (lengths is not None and lengths.shape != (B,)):
        raise ValueError("start and lengths must be [B]")
    od = out_dtype or v.dtype
    if out is None:
        out = (torch.empty if lengths is None else torch.zeros)((B, S, HV, V), dtype=od, device=dev)
    else:
        out = _output(out, "out", (B, S, HV, V), od, dev)
    _call(_load().kda_gdr_recurrent_step, dev, _p(q), _p(k), _p(v), _dtype_code(q.dtype), _p(g), 1 if g.dim() == 4 else 0, _p(beta), _p(states),
          pool, _p(slots), cols, _p(start), _p(lengths), B, S, HK, HV, K, V, float(scale), _p(out), _dtype_code(od))
    return out


def draft_verify(target_probs: torch.Tensor, draft_tokens: torch.Tensor, uniforms: torch.Tensor,
                 draft_probs: Optional[torch.Tensor] = None, lengths: Optional[torch.Tensor] = None
                 ) -> Tuple[torch.Tensor, torch.Tensor]:
    """The drafted tokens of B requests against the target's probabilities.  target_probs
    [B,D+1,vocab] float32; draft_tokens int32 [B,D]; draft_probs [B,D,vocab] float32, what the
    drafts were drawn from (None: each was certain); uniforms [B,D+1] float32 in [0, 1): one for
    each draft, and one to draw with; lengths int32 [B]: drafts of each request (None: D).

    Draft i holds while u_i q_i(x_i) < p_i(x_i).  Behind the last that holds one token is drawn,
    from max(p - q, 0) where a draft was refused (from p if that is nothing), from p where none
    was; in whole weights of 2^-44, so that no order of summation changes it.  A uniform of 1 or
    more draws the last token that has weight, NaN or one below 0 the first.  Returns (tokens
    int32 [B,D+1]: the drafts that hold, the token drawn, then -1; accepted int32 [B])."""
    p = _input(target_probs, "target_probs", None, torch.float32, 4)
    if p is None:
        raise TypeError("target_probs must be a torch.Tensor")
    x, u = _input(draft_tokens, "draft_tokens", p, torch.int32, 4), _input(uniforms, "uniforms", p, torch.float32, 4)
    q, lengths = _input(draft_probs, "draft_probs", p, torch.float32, 4), _input(lengths, "lengths", p, torch.int32, 4)
    if p.dim() != 3 or p.shape[1] < 1:
        raise ValueError("target_probs must be [B, D + 1, vocab]")
    B, D, vocab = p.shape[0], p.shape[1] - 1, p.shape[2]
    if x.shape != (B, D) or u.shape != (B, D + 1) or (q is not None and q.shape != (B, D, vocab)) or (
            lengths is not None and lengths.shape != (B,)):
        raise ValueError("draft_tokens must be [B, D], uniforms [B, D + 1], draft_probs [B, D, vocab] and lengths [B]")
    dev = p.device
    tokens = torch.empty((B, D + 1), dtype=torch.int32, device=dev)
    accepted = torch.empty((B,), dtype=torch.int32, device=dev)
    workspace = _workspace(None, _workspace_size("kda_draft_verify_workspace_size", B, vocab), dev)
    _call(_load().kda_draft_verify, dev, _p(p), _p(x), _p(q), _p(u), _p(lengths), B, D, vocab, _p(tokens), _p(accepted), _p(workspace),
          workspace.numel())
    return tokens, accepted
