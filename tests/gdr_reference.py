"""Plain 64-bit forms of the gated delta rule with one decay per value head and of decoding
with drafted tokens, for the tests: the scan goes token by token through the fp64 oracle
(heads repeated over their group, a head's decay over its channels), the verification is a
loop over whole numbers."""
from __future__ import annotations

import math

import numpy as np
import torch

import oracle
from tests.helpers import f64


def make(B, T, HK, HV, K, V, dtype=torch.float32, seed=0, seqlens=None, state=True, decay=(0.02, 4.0)):
    """Inputs as a layer makes them; a head's decays are scaled by a rate of its own in `decay`."""
    gen = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True).clamp_min(1e-6)  # noqa: E731
    q, k = (unit(torch.nn.functional.silu(rand(B, T, HK, K))).to(dtype) for _ in range(2))
    v = torch.nn.functional.silu(rand(B, T, HV, V)).to(dtype)
    lo, hi = (math.log(x) for x in decay)
    g = -torch.nn.functional.softplus(rand(B, T, HV)) * torch.exp(lo + (hi - lo) * torch.rand(HV, generator=gen))
    beta = torch.sigmoid(rand(B, T, HV))
    cu = None if seqlens is None else torch.tensor(np.concatenate([[0], np.cumsum(seqlens)]), dtype=torch.int32)
    N = B if seqlens is None else len(seqlens)
    s0 = 0.3 * rand(N, HV, K, V) if state else None
    return dict(q=q, k=k, v=v, g=g, beta=beta, s0=s0, cu=cu, N=N)


def repeated(x, HV):
    return np.repeat(f64(x), HV // x.shape[2], axis=2)


def scan(i, scale=1.0):
    """(out, final state) of make()'s inputs."""
    HV, K = i["v"].shape[2], i["q"].shape[3]
    alpha = np.repeat(np.exp(f64(i["g"]))[..., None], K, axis=3)
    cu = None if i["cu"] is None else f64(i["cu"]).astype(np.int64)
    return oracle.scan(repeated(i["q"], HV), repeated(i["k"], HV), f64(i["v"]), alpha, f64(i["beta"]),
                       None if i["s0"] is None else f64(i["s0"]), cu_seqlens=cu, scale=scale)


def scan_bwd(i, d_out, d_final, scale=1.0):
    """Gradients (dq, dk, dv, dg, dbeta, ds0): the oracle's, summed over a group's heads and a head's channels."""
    HK, HV, K = i["q"].shape[2], i["v"].shape[2], i["q"].shape[3]
    alpha = np.repeat(np.exp(f64(i["g"]))[..., None], K, axis=3)
    cu = None if i["cu"] is None else f64(i["cu"]).astype(np.int64)
    dq, dk, dv, da, db, ds = oracle.scan_bwd(repeated(i["q"], HV), repeated(i["k"], HV), f64(i["v"]), alpha, f64(i["beta"]), f64(d_out),
                                             None if i["s0"] is None else f64(i["s0"]), None if d_final is None else f64(d_final),
                                             cu_seqlens=cu, scale=scale)
    B, T = dq.shape[:2]
    shared = lambda x: x.reshape(B, T, HK, HV // HK, K).sum(3)  # noqa: E731
    return shared(dq), shared(dk), dv, (da * alpha).sum(-1), db, ds


def step(q, k, v, g, beta, states, slots, start, lengths, scale=1.0):
    """gdr_recurrent_step on float64 copies: (out with NaN in the rows that are not written, states)."""
    B, S, HV = beta.shape
    q, k, v, g, beta, states = repeated(q, HV), repeated(k, HV), f64(v), f64(g), f64(beta), f64(states).copy()
    out = np.full((B, S, HV, v.shape[-1]), np.nan)
    before = states.copy()
    cols, pool = slots.shape[1], len(states)
    for b in range(B):
        c = 0 if start is None else int(start[b])
        at = int(slots[b, c]) if 0 <= c < cols else -1
        x = before[at].copy() if 0 <= at < pool else np.zeros(states.shape[1:])
        n = S if lengths is None else min(max(int(lengths[b]), 0), S)
        for t in range(n):
            a = np.exp(g[b, t])
            x = x * (a[..., None] if a.ndim == 2 else a[:, None, None])
            d = beta[b, t][:, None] * (v[b, t] - np.einsum("hkv,hk->hv", x, k[b, t]))
            x = x + k[b, t][..., None] * d[:, None, :]
            out[b, t] = scale * np.einsum("hkv,hk->hv", x, q[b, t])
            to = int(slots[b, t]) if cols > 1 else int(slots[b, 0]) if t == n - 1 else -1
            if 0 <= to < pool:
                states[to] = x
    return out, states


def verify(p, x, u, q=None, lengths=None):
    """draft_verify, one request after another, in Python's own whole numbers."""
    p, u = f64(p), f64(u)
    q = None if q is None else f64(q)
    B, D1, vocab = p.shape
    tokens, accepted = np.full((B, D1), -1, dtype=np.int32), np.zeros(B, dtype=np.int32)
    whole = lambda w: np.floor(np.clip(np.nan_to_num(w, nan=0.0, posinf=1.0, neginf=0.0), 0, 1) * 2.0 ** 44).astype(np.int64)  # noqa: E731
    for b in range(B):
        n = D1 - 1 if lengths is None else min(max(int(lengths[b]), 0), D1 - 1)
        a = 0
        while a < n:
            t = int(x[b, a])
            if not 0 <= t < vocab or not u[b, a] * (1.0 if q is None else q[b, a, t]) < p[b, a, t]:
                break
            tokens[b, a] = t
            a += 1
        off = np.zeros(vocab)
        if a < n:
            if q is not None:
                off = q[b, a]
            elif 0 <= int(x[b, a]) < vocab:
                off[int(x[b, a])] = 1.0
        w = whole(p[b, a] - off)
        if w.sum() == 0:
            w = whole(p[b, a])
        c = np.cumsum(w)
        t = min(int(u[b, -1] * float(c[-1])), int(c[-1]) - 1)
        tokens[b, a] = int(np.sum(c <= t))
        accepted[b] = a
    return tokens, accepted
