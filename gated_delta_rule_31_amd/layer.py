"""What stands around the recurrence in a layer: the short convolution, the gated linear recurrence, the norms.

* ``short_conv_fwd(x, weight, ...)`` -- the short causal convolution (and silu) of a layer's rows,
  over packed sequences and kept rows; ``short_conv_bwd`` -- its gradients; ``short_conv(...)`` --
  recorded for autograd; ``short_conv_step`` -- decoding over a pool of kept rows.
* ``glr_fwd(x, gate, ...)`` -- the gated linear recurrence h_t = alpha_t h_{t-1} + f_t sigmoid(i_t)
  x_t of every channel, alpha the bounded decay of logits or given as log decays; ``glr_bwd`` --
  its gradients; ``gated_linear_recurrence(...)`` -- recorded; ``glr_step`` -- decoding over a
  pool of states.
* ``block_norm_fwd(y, ...)`` -- norm behind a block, gate, residual scale, residual and norm before
  the next block in one call; ``block_norm_bwd`` -- its gradients; ``block_norm(...)`` -- recorded;
  ``gated_norm(y, gate, weight)`` -- a recurrence's heads: norm and gate alone, recorded.

Sequences of a packed batch do not reach each other, whatever they hold.  Forward-mode derivatives are refused, as
everywhere in the library.

The decode calls take ``slots``, ``start`` and ``lengths`` as ``gdr_recurrent_step`` does, so that a
layer's convolution, recurrence and drafts go by one table.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import _dtype_code, _load, _needs_grad
from .gdr import _call, _input, _output, _p, _workspace, _workspace_size

SILU = 8                           # flags of the C calls
NORMALIZE = 1
NORM_AFTER, NORM_BEFORE = 1, 2


def _rows(x: Optional[torch.Tensor], name: str, like: Optional[torch.Tensor] = None, dtype=None) -> Tuple[Optional[torch.Tensor], int]:
    """A tensor [B, T, ...] as rows that are dense each and lie at one distance from one another (copied if
    need be), and that distance."""
    if x is None:
        return None, 0
    if isinstance(x, torch.Tensor) and x.dim() >= 2 and x.numel() and not x.is_contiguous():
        width, dense, stride = 1, True, x.stride(1) if x.shape[1] > 1 else x.stride(0)
        for n, s in zip(reversed(x.shape[2:]), reversed(x.stride()[2:])):
            dense, width = dense and (n == 1 or s == width), width * n
        if dense and stride >= width and (x.shape[0] == 1 or x.shape[1] == 1 or x.stride(0) == x.shape[1] * stride):
            return _input_view(x, name, like, dtype), stride
    x = _input(x, name, like, dtype, 1)
    return x, x.shape[2:].numel() if x.dim() > 2 else 1


def _input_view(x, name, like, dtype):
    """The checks of ``_input`` for a tensor that is taken with its strides."""
    _input(x[:1, :1], name, like, dtype, 1)
    return x


def _like(x: Optional[torch.Tensor], name: str, like: torch.Tensor, dtype, shape) -> Optional[torch.Tensor]:
    x = _input(x, name, like, dtype, 1)
    if x is not None and tuple(x.shape) != tuple(shape):
        raise ValueError("%s must be %s (got %s)" % (name, list(shape), list(x.shape)))
    return x


def _sequences(cu_seqlens, like, B):
    cu_seqlens = _input(cu_seqlens, "cu_seqlens", like, torch.int32, 4)
    if cu_seqlens is not None and (cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1):
        raise ValueError("cu_seqlens must be int32 [N + 1]")
    return cu_seqlens, B if cu_seqlens is None else cu_seqlens.numel() - 1


def _made(x, name, shape, dtype, device):
    return torch.empty(shape, dtype=dtype, device=device) if x is None else _output(x, name, shape, dtype, device)


def _pool(slots, start, lengths, like, states, B, S):
    slots, start, lengths = (_input(x, n, like, torch.int32, 4) for x, n in ((slots, "slots"), (start, "start"), (lengths, "lengths")))
    cols = 1
    if slots is not None:
        cols = 1 if slots.dim() == 1 else slots.shape[-1]
        if slots.dim() not in (1, 2) or slots.shape[0] != B or cols not in (1, S):
            raise ValueError("slots must be [B], [B, 1] or [B, S]")
    if slots is None and (start is not None or states.shape[0] < B):
        raise ValueError("without slots every request has a state of its own, states[b], and starts from it")
    if start is not None and cols != S:
        raise ValueError("start names a column of slots [B, S]")
    if (start is not None and start.shape != (B,)) or (lengths is not None and lengths.shape != (B,)):
        raise ValueError("start and lengths must be [B]")
    return slots, start, lengths, cols


def _step_out(out, lengths, x):
    if out is None:
        return (torch.empty if lengths is None else torch.zeros)(x.shape, dtype=x.dtype, device=x.device)
    return _output(out, "out", x.shape, x.dtype, x.device)


# --------------------------------------------------------------------------- the short convolution

def _conv_inputs(x, weight, bias, initial_state, cu_seqlens):
    x, stride = _rows(x, "x")
    if x is None:
        raise TypeError("x must be a torch.Tensor")
    if x.dim() != 3:
        raise ValueError("x must be [B, T, D]")
    B, T, D = x.shape
    weight = _input(weight, "weight", x, torch.float32, 4)
    if weight is None or weight.dim() != 2 or weight.shape[0] != D:
        raise ValueError("weight must be [D, W]")
    W = weight.shape[1]
    bias = _like(bias, "bias", x, torch.float32, (D,))
    cu_seqlens, N = _sequences(cu_seqlens, x, B)
    initial_state = _like(initial_state, "initial_state", x, x.dtype, (N, W - 1, D))
    return x, stride, weight, bias, initial_state, cu_seqlens, (B, T, D, W, N)


def short_conv_fwd(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None, initial_state: Optional[torch.Tensor] = None,
                   output_final_state: bool = True, cu_seqlens: Optional[torch.Tensor] = None, silu: bool = True,
                   out: Optional[torch.Tensor] = None, final_state: Optional[torch.Tensor] = None
                   ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """out_t = silu(bias + sum_w weight[:, w] x_{t - W + 1 + w}) (without silu the sum itself).  x [B,T,D]
    float32 or bfloat16, rows dense, a slice of a wider tensor without a copy; weight [D,W] float32, W in
    2..4, the last column the row's own; bias [D] float32; initial_state [N,W-1,D] like x, the rows
    before each sequence, oldest first (None: zeros); cu_seqlens int32 [N+1] (B == 1) or None.
    Returns (out [B,T,D], final_state [N,W-1,D], the last rows of each sequence, or None).  Rows of
    ``out`` behind the last packed sequence are left as they were (unset in an ``out`` made here)."""
    x, stride, weight, bias, initial_state, cu_seqlens, (B, T, D, W, N) = _conv_inputs(x, weight, bias, initial_state, cu_seqlens)
    out = _made(out, "out", (B, T, D), x.dtype, x.device)
    if final_state is not None or output_final_state:
        final_state = _made(final_state, "final_state", (N, max(W - 1, 0), D), x.dtype, x.device)
    _call(_load().kda_short_conv_fwd, x.device, _p(x), stride, _dtype_code(x.dtype), _p(weight), _p(bias), _p(initial_state), _p(final_state),
          _p(cu_seqlens), N, B, T, D, W, SILU if silu else 0, _p(out))
    return out, final_state


def short_conv_bwd_workspace_size(dtype: torch.dtype, B: int, T: int, D: int, W: int) -> int:
    """Bytes of device workspace ``short_conv_bwd`` needs for this shape (0: unsupported or empty)."""
    return _workspace_size("kda_short_conv_bwd_workspace_size", _dtype_code(dtype), int(B), int(T), int(D), int(W))


def short_conv_bwd(x: torch.Tensor, weight: torch.Tensor, d_out: torch.Tensor, bias: Optional[torch.Tensor] = None,
                   initial_state: Optional[torch.Tensor] = None, d_final_state: Optional[torch.Tensor] = None,
                   cu_seqlens: Optional[torch.Tensor] = None, silu: bool = True, want_d_initial_state: bool = True,
                   workspace: Optional[torch.Tensor] = None):
    """Gradients of ``short_conv_fwd`` for L = <d_out, out> + <d_final_state, final_state>: (dx, d_weight,
    d_bias (None without a bias), d_initial_state or None), dx and d_initial_state like x, the others
    float32.  Rows behind the last packed sequence get zeros."""
    x, stride, weight, bias, initial_state, cu_seqlens, (B, T, D, W, N) = _conv_inputs(x, weight, bias, initial_state, cu_seqlens)
    d_out = _like(d_out, "d_out", x, x.dtype, (B, T, D))
    if d_out is None:
        raise TypeError("d_out must be a torch.Tensor")
    d_final_state = _like(d_final_state, "d_final_state", x, x.dtype, (N, W - 1, D))
    dev = x.device
    dx, dw = torch.empty((B, T, D), dtype=x.dtype, device=dev), torch.empty((D, W), dtype=torch.float32, device=dev)
    db = torch.empty((D,), dtype=torch.float32, device=dev) if bias is not None else None
    ds = torch.empty((N, W - 1, D), dtype=x.dtype, device=dev) if want_d_initial_state else None
    workspace = _workspace(workspace, short_conv_bwd_workspace_size(x.dtype, B, T, D, W), dev)
    _call(_load().kda_short_conv_bwd, dev, _p(x), stride, _dtype_code(x.dtype), _p(weight), _p(bias), _p(initial_state), _p(cu_seqlens), N, B, T, D,
          W, SILU if silu else 0, _p(d_out), _p(d_final_state), _p(dx), _p(dw), _p(db), _p(ds), _p(workspace), workspace.numel())
    return dx, dw, db, ds


def short_conv_step(x: torch.Tensor, weight: torch.Tensor, states: torch.Tensor, bias: Optional[torch.Tensor] = None,
                    slots: Optional[torch.Tensor] = None, start: Optional[torch.Tensor] = None, lengths: Optional[torch.Tensor] = None,
                    silu: bool = True, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Up to S tokens for each of B requests over a pool of kept rows: x [B,S,D], states [pool,W-1,D] like
    x, contiguous, updated in place.  ``slots``, ``start`` and ``lengths`` as in ``gdr_recurrent_step``.
    Returns out [B,S,D]."""
    x = _input(x, "x", None, None, 1)
    if x is None or x.dim() != 3:
        raise ValueError("x must be [B, S, D]")
    B, S, D = x.shape
    weight = _input(weight, "weight", x, torch.float32, 4)
    if weight is None or weight.dim() != 2 or weight.shape[0] != D:
        raise ValueError("weight must be [D, W]")
    W = weight.shape[1]
    bias = _like(bias, "bias", x, torch.float32, (D,))
    if not isinstance(states, torch.Tensor) or states.dim() != 3:
        raise ValueError("states must be [pool, W - 1, D]")
    states = _output(states, "states", (states.shape[0], W - 1, D), x.dtype, x.device)
    slots, start, lengths, cols = _pool(slots, start, lengths, x, states, B, S)
    out = _step_out(out, lengths, x)
    _call(_load().kda_short_conv_step, x.device, _p(x), _dtype_code(x.dtype), _p(weight), _p(bias), _p(states), states.shape[0], _p(slots), cols,
          _p(start), _p(lengths), B, S, D, W, SILU if silu else 0, _p(out))
    return out


def _d(x):
    return None if x is None else x.detach()


class _ShortConvFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, initial_state, cu_seqlens, silu):
        with torch.no_grad():
            out, final = _conv_zeros_behind(_d(x), _d(weight), _d(bias), _d(initial_state), cu_seqlens, silu)
        ctx.save_for_backward(x, weight, bias, initial_state, cu_seqlens)
        ctx.silu = silu
        ctx.set_materialize_grads(False)
        return out, final

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, d_out, d_final):
        x, weight, bias, s0, cu = ctx.saved_tensors
        if d_out is None:
            d_out = torch.zeros(x.shape, dtype=x.dtype, device=x.device)
        with torch.no_grad():
            dx, dw, db, ds = short_conv_bwd(_d(x), _d(weight), d_out, bias=_d(bias), initial_state=_d(s0), d_final_state=d_final, cu_seqlens=cu,
                                            silu=ctx.silu, want_d_initial_state=ctx.needs_input_grad[3])
        return dx, dw, db, ds, None, None


def _conv_zeros_behind(x, weight, bias, initial_state, cu_seqlens, silu):
    out = None if cu_seqlens is None else torch.zeros(x.shape, dtype=x.dtype, device=x.device)
    return short_conv_fwd(x, weight, bias=bias, initial_state=initial_state, cu_seqlens=cu_seqlens, silu=silu, out=out)


def short_conv(x, weight, bias=None, initial_state=None, cu_seqlens=None, silu: bool = True):
    """``short_conv_fwd`` as a function of its inputs: (out, final_state), recorded for autograd when any of x,
    weight, bias or initial_state requires grad.  Rows of out behind the last packed sequence are zeros."""
    if _needs_grad(x, weight, bias, initial_state):
        return _ShortConvFn.apply(x, weight, bias, initial_state, cu_seqlens, bool(silu))
    return _conv_zeros_behind(x, weight, bias, initial_state, cu_seqlens, silu)


# --------------------------------------------------------------------------- the gated linear recurrence

def _glr_inputs(x, gate, log_scale, bias, in_gate):
    x, x_stride = _rows(x, "x")
    if x is None:
        raise TypeError("x must be a torch.Tensor")
    if x.dim() != 4:
        raise ValueError("x must be [B, T, H, K]")
    H, K = x.shape[2:]
    log_scale = _like(log_scale, "log_scale", x, torch.float32, (H,))
    bias = _input(bias, "bias", x, torch.float32, 4)
    if bias is not None and (log_scale is None or bias.numel() != H * K):
        raise ValueError("bias must be [H, K], and goes with log_scale")
    gate, gate_stride = _rows(gate, "gate", x, torch.float32 if log_scale is None else x.dtype)
    in_gate, in_stride = _rows(in_gate, "in_gate", x, x.dtype)
    if gate is None:
        raise TypeError("gate must be a torch.Tensor")
    if gate.shape != x.shape or (in_gate is not None and in_gate.shape != x.shape):
        raise ValueError("gate and in_gate must be shaped like x")
    return x, x_stride, gate, gate_stride, log_scale, bias, in_gate, in_stride


def glr_kept_size(B: int, T: int, H: int, K: int) -> int:
    """Bytes of what ``glr_fwd`` keeps for ``glr_bwd`` (``keep=True``)."""
    return _workspace_size("kda_glr_kept_size", int(B), int(T), int(H), int(K))


def glr_fwd_workspace_size(B: int, T: int, H: int, K: int) -> int:
    """Bytes of device workspace ``glr_fwd`` needs for this shape (0: unsupported or empty)."""
    return _workspace_size("kda_glr_fwd_workspace_size", int(B), int(T), int(H), int(K))


def glr_fwd(x: torch.Tensor, gate: torch.Tensor, log_scale: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
            in_gate: Optional[torch.Tensor] = None, initial_state: Optional[torch.Tensor] = None, output_final_state: bool = True,
            cu_seqlens: Optional[torch.Tensor] = None, lower_bound: float = -5.0, normalize: bool = True, keep: bool = False,
            out: Optional[torch.Tensor] = None, final_state: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """h_t = alpha_t h_{t-1} + f_t sigmoid(in_gate_t) x_t for every channel, out_t = h_t; f = sqrt(1 - alpha^2)
    with ``normalize``, else 1; without in_gate the input as it is.  x, in_gate [B,T,H,K] float32 or
    bfloat16, rows dense, slices of wider tensors without a copy.  gate [B,T,H,K]: with log_scale [H]
    float32 (and bias [H,K]) logits in the type of x, alpha = exp(lower_bound sigmoid(exp(log_scale)
    (gate + bias))) as ``bounded_decay`` has it; without log_scale ln alpha itself, float32, <= 0.
    initial_state [N,H,K] float32 or None (zeros); cu_seqlens int32 [N+1] (B == 1) or None.  Returns
    (out [B,T,H,K] like x, final_state [N,H,K] float32 or None), and with ``keep`` a third: what
    ``glr_bwd`` would make again.  Rows of ``out`` behind the last packed sequence are left as they were."""
    x, x_stride, gate, gate_stride, log_scale, bias, in_gate, in_stride = _glr_inputs(x, gate, log_scale, bias, in_gate)
    B, T, H, K = x.shape
    cu_seqlens, N = _sequences(cu_seqlens, x, B)
    initial_state = _like(initial_state, "initial_state", x, torch.float32, (N, H, K))
    dev = x.device
    out = _made(out, "out", (B, T, H, K), x.dtype, dev)
    if final_state is not None or output_final_state:
        final_state = _made(final_state, "final_state", (N, H, K), torch.float32, dev)
    kept = torch.empty(glr_kept_size(B, T, H, K) // 4, dtype=torch.float32, device=dev) if keep else None
    workspace = _workspace(workspace, glr_fwd_workspace_size(B, T, H, K), dev)
    _call(_load().kda_glr_fwd, dev, _p(x), x_stride, _dtype_code(x.dtype), _p(gate), gate_stride, _p(log_scale), _p(bias), float(lower_bound),
          _p(in_gate), in_stride, NORMALIZE if normalize else 0, _p(initial_state), _p(final_state), _p(cu_seqlens), N, B, T, H, K, _p(out), _p(kept),
          _p(workspace), workspace.numel())
    return (out, final_state, kept) if keep else (out, final_state)


def glr_bwd_workspace_size(B: int, T: int, H: int, K: int, logits: bool = True, kept: bool = True) -> int:
    """Bytes of device workspace ``glr_bwd`` needs for this shape (0: unsupported or empty)."""
    return _workspace_size("kda_glr_bwd_workspace_size", int(B), int(T), int(H), int(K), 1 if logits else 0, 1 if kept else 0)


def glr_bwd(x: torch.Tensor, gate: torch.Tensor, d_out: torch.Tensor, log_scale: Optional[torch.Tensor] = None,
            bias: Optional[torch.Tensor] = None, in_gate: Optional[torch.Tensor] = None, initial_state: Optional[torch.Tensor] = None,
            d_final_state: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None, lower_bound: float = -5.0,
            normalize: bool = True, kept: Optional[torch.Tensor] = None, want_d_initial_state: bool = True,
            workspace: Optional[torch.Tensor] = None):
    """Gradients of ``glr_fwd`` (same inputs) for L = <d_out, out> + <d_final_state, final_state>: (dx, d_gate,
    d_in_gate, d_log_scale, d_bias, d_initial_state), each like what it is the gradient of (float32
    for the last three; None for what was not given).  ``kept``: the third of what ``glr_fwd(...,
    keep=True)`` returned for the same inputs; without it the states are made again.  Rows behind the
    last packed sequence get zeros.  Infinite logits have the gradients of large ones (0)."""
    x, x_stride, gate, gate_stride, log_scale, bias, in_gate, in_stride = _glr_inputs(x, gate, log_scale, bias, in_gate)
    B, T, H, K = x.shape
    cu_seqlens, N = _sequences(cu_seqlens, x, B)
    initial_state = _like(initial_state, "initial_state", x, torch.float32, (N, H, K))
    d_final_state = _like(d_final_state, "d_final_state", x, torch.float32, (N, H, K))
    d_out = _like(d_out, "d_out", x, x.dtype, (B, T, H, K))
    if d_out is None:
        raise TypeError("d_out must be a torch.Tensor")
    kept = _like(kept, "kept", x, torch.float32, (glr_kept_size(B, T, H, K) // 4,))
    dev = x.device
    made = lambda like, dtype: None if like is None else torch.empty(like.shape, dtype=dtype, device=dev)  # noqa: E731
    dx, dg, di = made(x, x.dtype), made(gate, gate.dtype), made(in_gate, x.dtype)
    da, db = made(log_scale, torch.float32), made(bias, torch.float32)
    ds = torch.empty((N, H, K), dtype=torch.float32, device=dev) if want_d_initial_state else None
    workspace = _workspace(workspace, glr_bwd_workspace_size(B, T, H, K, log_scale is not None, kept is not None), dev)
    _call(_load().kda_glr_bwd, dev, _p(x), x_stride, _dtype_code(x.dtype), _p(gate), gate_stride, _p(log_scale), _p(bias), float(lower_bound),
          _p(in_gate), in_stride, NORMALIZE if normalize else 0, _p(initial_state), _p(cu_seqlens), N, B, T, H, K, _p(kept), _p(d_out),
          _p(d_final_state), _p(dx), _p(dg), _p(di), _p(da), _p(db), _p(ds), _p(workspace), workspace.numel())
    return dx, dg, di, da, db, ds


def glr_step(x: torch.Tensor, gate: torch.Tensor, states: torch.Tensor, log_scale: Optional[torch.Tensor] = None,
             bias: Optional[torch.Tensor] = None, in_gate: Optional[torch.Tensor] = None, slots: Optional[torch.Tensor] = None,
             start: Optional[torch.Tensor] = None, lengths: Optional[torch.Tensor] = None, lower_bound: float = -5.0,
             normalize: bool = True, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Up to S tokens for each of B requests over a pool of states: x, gate, in_gate [B,S,H,K] and their
    companions as in ``glr_fwd``, states [pool,H,K] float32 contiguous, updated in place.  ``slots``,
    ``start`` and ``lengths`` as in ``gdr_recurrent_step``.  Returns out [B,S,H,K]."""
    x, gate, in_gate = (y.contiguous() if isinstance(y, torch.Tensor) else y for y in (x, gate, in_gate))
    x, _, gate, _, log_scale, bias, in_gate, _ = _glr_inputs(x, gate, log_scale, bias, in_gate)
    B, S, H, K = x.shape
    if not isinstance(states, torch.Tensor) or states.dim() != 3:
        raise ValueError("states must be [pool, H, K]")
    states = _output(states, "states", (states.shape[0], H, K), torch.float32, x.device)
    slots, start, lengths, cols = _pool(slots, start, lengths, x, states, B, S)
    out = _step_out(out, lengths, x)
    _call(_load().kda_glr_step, x.device, _p(x), _dtype_code(x.dtype), _p(gate), _p(log_scale), _p(bias), float(lower_bound), _p(in_gate),
          NORMALIZE if normalize else 0, _p(states), states.shape[0], _p(slots), cols, _p(start), _p(lengths), B, S, H, K, _p(out))
    return out


class _GlrFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gate, log_scale, bias, in_gate, initial_state, cu_seqlens, lower_bound, normalize):
        with torch.no_grad():
            out, final, kept = _glr_zeros_behind(_d(x), _d(gate), _d(log_scale), _d(bias), _d(in_gate), _d(initial_state), cu_seqlens, lower_bound,
                                                 normalize, True)
        ctx.save_for_backward(x, gate, log_scale, bias, in_gate, initial_state, cu_seqlens, kept)
        ctx.lower_bound, ctx.normalize = lower_bound, normalize
        ctx.set_materialize_grads(False)
        return out, final

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, d_out, d_final):
        x, gate, log_scale, bias, in_gate, s0, cu, kept = ctx.saved_tensors
        if d_out is None:
            d_out = torch.zeros(x.shape, dtype=x.dtype, device=x.device)
        with torch.no_grad():
            grads = glr_bwd(_d(x), _d(gate), d_out, log_scale=_d(log_scale), bias=_d(bias), in_gate=_d(in_gate), initial_state=_d(s0),
                            d_final_state=d_final, cu_seqlens=cu, lower_bound=ctx.lower_bound, normalize=ctx.normalize, kept=kept,
                            want_d_initial_state=ctx.needs_input_grad[5])
        dx, dg, di, da, db, ds = grads
        return dx, dg, da, db, di, ds, None, None, None


def _glr_zeros_behind(x, gate, log_scale, bias, in_gate, initial_state, cu_seqlens, lower_bound, normalize, keep=False):
    out = None if cu_seqlens is None else torch.zeros(x.shape, dtype=x.dtype, device=x.device)
    return glr_fwd(x, gate, log_scale=log_scale, bias=bias, in_gate=in_gate, initial_state=initial_state, cu_seqlens=cu_seqlens,
                   lower_bound=lower_bound, normalize=normalize, keep=keep, out=out)


def gated_linear_recurrence(x, gate, log_scale=None, bias=None, in_gate=None, initial_state=None, cu_seqlens=None, lower_bound: float = -5.0,
                            normalize: bool = True):
    """``glr_fwd`` as a function of its inputs: (out, final_state), recorded for autograd when any of them
    requires grad.  Rows of out behind the last packed sequence are zeros."""
    if _needs_grad(x, gate, log_scale, bias, in_gate, initial_state):
        return _GlrFn.apply(x, gate, log_scale, bias, in_gate, initial_state, cu_seqlens, float(lower_bound), bool(normalize))
    return _glr_zeros_behind(x, gate, log_scale, bias, in_gate, initial_state, cu_seqlens, lower_bound, normalize)


# --------------------------------------------------------------------------- norms between blocks

def _tokens_heads(shape):
    """[..., D] as tokens of heads: the dimension before the last is a token's heads where there are three or more."""
    n = 1
    for s in shape[:-1]:
        n *= s
    heads = shape[-2] if len(shape) > 2 and n else 1
    return n // heads, heads


def _gate_rows(gate, y, tokens, heads):
    """The gate, and the distances between its tokens and between a token's heads; one that is a slice of a wider
    tensor, tokens at one distance, is not copied."""
    if gate is None:
        return None, 0, 0
    if isinstance(gate, torch.Tensor) and gate.shape != y.shape:
        raise ValueError("gate must be shaped like y")
    D = y.shape[-1]
    if isinstance(gate, torch.Tensor) and gate.dim() >= 2 and gate.numel() and not gate.is_contiguous():
        lead, strides = (gate.shape[:-2], gate.stride()[:-2]) if gate.dim() > 2 else (gate.shape[:1], gate.stride()[:1])
        head = gate.stride(-2) if heads > 1 else D
        dense, stride, n = (D == 1 or gate.stride(-1) == 1) and head >= D, None, 1
        for size, s in zip(reversed(lead), reversed(strides)):
            if size > 1:
                stride = s if stride is None else stride
                dense = dense and s == stride * n
                n *= size
        stride = heads * D if stride is None else stride
        if dense and stride >= D:
            _input(gate[tuple(slice(0, 1) for _ in range(gate.dim()))], "gate", y, y.dtype, 1)
            return gate, stride, head
    return _input(gate, "gate", y, y.dtype, 1), heads * D, D


def _norm_inputs(y, gate, weight_after, weight_before, norm_after, norm_before, silu):
    y = _input(y, "y", None, None, 1)
    if y is None:
        raise TypeError("y must be a torch.Tensor")
    if y.dim() < 2 or y.shape[-1] < 1:
        raise ValueError("y must be [tokens, D] or [..., heads, D]")
    tokens, heads = _tokens_heads(y.shape)
    gate, *gate_strides = _gate_rows(gate, y, tokens, heads)
    weight_after = _like(weight_after, "weight_after", y, torch.float32, y.shape[-1:])
    weight_before = _like(weight_before, "weight_before", y, torch.float32, y.shape[-1:])
    flags = (NORM_AFTER if norm_after else 0) | (NORM_BEFORE if norm_before else 0) | (SILU if silu else 0)
    return y, gate, gate_strides, weight_after, weight_before, flags, (tokens, heads, y.shape[-1])


def block_norm_fwd(y: torch.Tensor, gate: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
                   weight_after: Optional[torch.Tensor] = None, weight_before: Optional[torch.Tensor] = None, norm_after: bool = True,
                   norm_before: bool = True, scale: float = 1.0, eps: float = 1e-6, silu: bool = False, out: Optional[torch.Tensor] = None
                   ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """A block's output y [..., D] on its way into the residual stream and the next block:
    p = y / rms(y) weight_after (``norm_after``; else y), h = residual + scale act(gate) p (act: sigmoid, or
    silu), n = h / rms(h) weight_before (``norm_before``), rms(x) = sqrt(mean x^2 + eps).  y, gate
    float32 or bfloat16 (the gate a slice of a wider tensor without a copy); residual like y or
    float32; weights [D] float32, None for ones.  The sums of a row's squares, of y and of h where they are
    normed, must be finite in float32.  Returns (h like the residual, or like y without
    one; n like y, or None).  ``out``: where h is written."""
    y, gate, gate_strides, weight_after, weight_before, flags, (tokens, heads, D) = _norm_inputs(y, gate, weight_after, weight_before, norm_after,
                                                                                               norm_before, silu)
    residual = _input(residual, "residual", y, None, 1)
    if residual is not None and residual.shape != y.shape:
        raise ValueError("residual must be shaped like y")
    h = _made(out, "out", y.shape, y.dtype if residual is None else residual.dtype, y.device)
    n = torch.empty(y.shape, dtype=y.dtype, device=y.device) if norm_before else None
    _call(_load().kda_block_norm_fwd, y.device, _p(y), _p(gate), *gate_strides, _dtype_code(y.dtype), _p(residual), _dtype_code(h.dtype),
          _p(weight_after), _p(weight_before), tokens, heads, D, float(scale), float(eps), flags, _p(h), _p(n))
    return h, n


def block_norm_bwd_workspace_size(tokens: int, heads: int, D: int) -> int:
    """Bytes of device workspace ``block_norm_bwd`` needs for this shape (0: unsupported or empty)."""
    return _workspace_size("kda_block_norm_bwd_workspace_size", int(tokens), int(heads), int(D))


def block_norm_bwd(y: torch.Tensor, d_h: Optional[torch.Tensor], d_n: Optional[torch.Tensor] = None, h: Optional[torch.Tensor] = None,
                   gate: Optional[torch.Tensor] = None, weight_after: Optional[torch.Tensor] = None,
                   weight_before: Optional[torch.Tensor] = None, norm_after: bool = True, norm_before: bool = True, scale: float = 1.0,
                   eps: float = 1e-6, silu: bool = False, workspace: Optional[torch.Tensor] = None):
    """Gradients of ``block_norm_fwd`` for L = <d_h, h> + <d_n, n>: (dy, d_gate, d_residual, d_weight_after,
    d_weight_before), None for what was not given.  h as the forward returned it, d_h like h (None:
    zeros) and d_n like y; without ``norm_before`` h and d_n are not used, and d_residual is d_h; without ``norm_after`` dy does not
    depend on y."""
    y, gate, gate_strides, weight_after, weight_before, flags, (tokens, heads, D) = _norm_inputs(y, gate, weight_after, weight_before, norm_after,
                                                                                               norm_before, silu)
    dev = y.device
    d_h = _input(d_h, "d_h", y, None, 1)
    if norm_before:
        h, d_n = _input(h, "h", y, None, 1), _like(d_n, "d_n", y, y.dtype, y.shape)
        if h is None or d_n is None or h.shape != y.shape:
            raise ValueError("norm_before needs h and d_n, shaped like y")
    elif d_h is None:
        raise ValueError("without norm_before d_h is what there is")
    like = h if norm_before else d_h
    if d_h is not None and (d_h.shape != y.shape or d_h.dtype != like.dtype):
        raise ValueError("d_h must be shaped like y, in the type of h")
    made = lambda x: None if x is None else torch.empty(x.shape, dtype=x.dtype, device=dev)  # noqa: E731
    dy, dz, dwa, dwb = made(y), made(gate), made(weight_after), made(weight_before)
    d_res = torch.empty(y.shape, dtype=like.dtype, device=dev) if norm_before else d_h
    workspace = _workspace(workspace, block_norm_bwd_workspace_size(tokens, heads, D), dev)
    _call(_load().kda_block_norm_bwd, dev, _p(y), _p(gate), *gate_strides, _dtype_code(y.dtype), _p(h) if norm_before else None,
          _dtype_code(like.dtype), _p(weight_after), _p(weight_before), tokens, heads, D, float(scale), float(eps), flags, _p(d_h),
          _p(d_n) if norm_before else None, _p(dy), _p(dz), _p(d_res) if norm_before else None, _p(dwa), _p(dwb), _p(workspace), workspace.numel())
    return dy, dz, d_res, dwa, dwb


class _BlockNormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, gate, residual, weight_after, weight_before, norm_after, norm_before, scale, eps, silu):
        with torch.no_grad():
            h, n = block_norm_fwd(_d(y), _d(gate), _d(residual), _d(weight_after), _d(weight_before), norm_after, norm_before, scale, eps, silu)
        ctx.save_for_backward(y, gate, weight_after, weight_before, h if norm_before else None)
        ctx.residual = residual is not None
        ctx.rest = norm_after, norm_before, scale, eps, silu
        ctx.set_materialize_grads(False)
        return h, n

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, d_h, d_n):
        y, gate, wa, wb, h = ctx.saved_tensors
        norm_after, norm_before, scale, eps, silu = ctx.rest
        if d_h is None and d_n is None:
            return (None,) * 10
        through = norm_before and d_n is not None
        with torch.no_grad():
            dy, dz, dr, dwa, dwb = block_norm_bwd(_d(y), d_h, d_n if through else None, _d(h) if through else None, _d(gate), _d(wa),
                                                  _d(wb) if through else None, norm_after, through, scale, eps, silu)
        if wb is not None and dwb is None:
            dwb = torch.zeros_like(wb)
        return dy, dz, dr if ctx.residual else None, dwa, dwb, None, None, None, None, None


def block_norm(y, gate=None, residual=None, weight_after=None, weight_before=None, norm_after: bool = True, norm_before: bool = True,
               scale: float = 1.0, eps: float = 1e-6, silu: bool = False):
    """``block_norm_fwd`` as a function of its inputs: (h, n), recorded for autograd when any of y, gate,
    residual or a weight requires grad."""
    if _needs_grad(y, gate, residual, weight_after, weight_before):
        return _BlockNormFn.apply(y, gate, residual, weight_after, weight_before, bool(norm_after), bool(norm_before), float(scale), float(eps),
                                  bool(silu))
    return block_norm_fwd(y, gate, residual, weight_after, weight_before, norm_after, norm_before, scale, eps, silu)


def gated_norm(y, gate=None, weight=None, eps: float = 1e-6, silu: bool = False):
    """A recurrence's heads y [..., D] behind it: y / rms(y) weight act(gate), recorded for autograd."""
    return block_norm(y, gate=gate, weight_after=weight, norm_before=False, eps=eps, silu=silu)[0]
