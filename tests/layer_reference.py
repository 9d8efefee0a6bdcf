"""Plain 64-bit forms of what stands around the recurrence in a layer, for the tests: differentiable, on
the CPU, one sequence after another and one row after another."""
from __future__ import annotations

import torch


def f64(x):
    return None if x is None else x.detach().to("cpu", torch.float64)


def rows_of(lens, packed):
    """(batch row, first row, length) of every sequence."""
    at, out = 0, []
    for i, n in enumerate(lens):
        out.append((0, at, n) if packed else (i, 0, n))
        at += n
    return out


def silu(x):
    return x * torch.sigmoid(x)


def conv(x, weight, bias, s0, lens, packed, act=True):
    """(out, final states); rows behind the last sequence are zeros."""
    W = weight.shape[1]
    out, finals = torch.zeros_like(x), []
    parts = []
    for i, (b, at, n) in enumerate(rows_of(lens, packed)):
        before = s0[i] if s0 is not None else x.new_zeros(W - 1, x.shape[2])
        rows = torch.cat([before, x[b, at : at + n]])
        finals.append(rows[n:])
        pre = sum(rows[j : j + n] * weight[:, j] for j in range(W)) + (bias if bias is not None else 0)
        parts.append((b, at, silu(pre) if act else pre))
    return _place(out, parts), torch.stack(finals) if finals else x.new_zeros(0, W - 1, x.shape[2])


def _place(out, parts):
    rows = [list(out[b].split(1)) for b in range(out.shape[0])]
    for b, at, y in parts:
        for t in range(y.shape[0]):
            rows[b][at + t] = y[t : t + 1]
    return torch.stack([torch.cat(r) if r else out[b] for b, r in enumerate(rows)]) if rows else out


def decay(gate, log_scale, bias, lower=-5.0):
    if log_scale is None:
        return gate
    z = gate if bias is None else gate + bias
    return lower * torch.sigmoid(torch.exp(log_scale)[:, None] * z)


def scan(x, gate, log_scale, bias, in_gate, s0, lens, packed, normalize=True, lower=-5.0):
    """(out, final states); rows behind the last sequence are zeros."""
    g = decay(gate, log_scale, bias, lower)
    a = torch.exp(g)
    u = x if in_gate is None else torch.sigmoid(in_gate) * x
    if normalize:
        u = u * torch.sqrt(-torch.expm1(2 * g))
    out, finals, parts = torch.zeros_like(x), [], []
    for i, (b, at, n) in enumerate(rows_of(lens, packed)):
        h = s0[i] if s0 is not None else x.new_zeros(x.shape[2:])
        ys = []
        for t in range(at, at + n):
            h = a[b, t] * h + u[b, t]
            ys.append(h)
        finals.append(h)
        parts.append((b, at, torch.stack(ys) if ys else x.new_zeros(0, *x.shape[2:])))
    return _place(out, parts), torch.stack(finals) if finals else x.new_zeros(0, *x.shape[2:])


def block_norm(y, gate, residual, wa, wb, after, before, scale, eps, act):
    rms = lambda x: torch.sqrt((x * x).mean(-1, keepdim=True) + eps)  # noqa: E731
    p = y
    if after:
        p = y / rms(y) * (wa if wa is not None else 1)
    if gate is not None:
        p = p * (silu(gate) if act else torch.sigmoid(gate))
    h = scale * p + (residual if residual is not None else 0)
    return h, (h / rms(h) * (wb if wb is not None else 1) if before else None)


def slots_walk(step, x, states, slots, start, lengths):
    """A decode call's order of reading and writing slots: `step(state, x_b_t, b, t)` gives (output, state).
    Rows that are not written are NaN."""
    B, S = x.shape[:2]
    cols, pool = slots.shape[1], states.shape[0]
    before, after, out = states, states.clone(), torch.full_like(x, float("nan"))
    for b in range(B):
        c = 0 if start is None else int(start[b])
        at = int(slots[b, c]) if 0 <= c < cols else -1
        s = before[at].clone() if 0 <= at < pool else torch.zeros_like(states[0])
        n = S if lengths is None else min(max(int(lengths[b]), 0), S)
        for t in range(n):
            out[b, t], s = step(s, x[b, t], b, t)
            to = int(slots[b, t]) if cols > 1 else int(slots[b, 0]) if t == n - 1 else -1
            if 0 <= to < pool:
                after[to] = s
    return out, after


def conv_token(weight, bias, act=True):
    def step(s, x, b, t):
        rows = torch.cat([s, x[None]])
        pre = (rows * weight.T).sum(0) + (bias if bias is not None else 0)
        return silu(pre) if act else pre, rows[1:]
    return step


def scan_token(gate, log_scale, bias, in_gate, normalize, lower=-5.0):
    g = decay(gate, log_scale, bias, lower)

    def step(s, x, b, t):
        u = x if in_gate is None else torch.sigmoid(in_gate[b, t]) * x
        u = u * torch.sqrt(-torch.expm1(2 * g[b, t])) if normalize else u
        h = torch.exp(g[b, t]) * s + u
        return h, h
    return step
