"""The operators around the recurrence in a layer: their cases, their plain forms in elementary
torch operations, and the calls that a user makes of the library.

* ``conv_*`` -- the short causal convolution of a layer's rows, channel by channel, over packed
  sequences and kept rows: prefill (``short_conv_fwd``), its gradients (``short_conv_bwd``) and
  decoding over a pool of kept rows (``short_conv_step``).  pre_t = bias + sum_w weight[:, w]
  x_{t - W + 1 + w}, out = silu(pre) or pre.
* ``scan_*`` -- the gated linear recurrence h_t = e^{g_t} h_{t-1} + s_t sigmoid(i_t) x_t of every
  channel, g the library's bounded decay of its logits or log decays as given, s = sqrt(1 - e^{2g})
  or 1: prefill (``glr_fwd``), forward and gradients (``glr_fwd``, ``glr_bwd``), decoding
  (``glr_step``).
* ``norm_*`` -- what stands between two blocks, or behind a recurrence's heads: p = rms(y) w_after,
  h = residual + scale act(gate) p, n = rms(h) w_before (``block_norm_fwd``, ``block_norm_bwd``).
"""
import math

import torch

own = False

LOWER, EPS = -5.0, 1e-6


# --------------------------------------------------------------------------- the cases

def listed():
    return [
        # q, k and v of a serving batch of one layer: packed prompts of ragged lengths, one of them empty, one of one token,
        # some going on from kept rows
        dict(name="conv prompts", op="conv_fwd", lens="3001,1,517,0,1024,64,1300,2049", packed=True, D=12288, W=4, dtype="bf16", silu=True, bias=False, s0=True, wide=True),
        # a training step's gradients over two rows
        dict(name="conv gradients", op="conv_bwd", lens="4096,4096", packed=False, D=4096, W=4, dtype="bf16", silu=True, bias=True, s0=False, wide=False),
        # decoding with drafts for a batch: the rows kept after every drafted token
        dict(name="conv drafts", op="conv_step", B=64, S=4, D=12288, W=4, dtype="bf16", silu=True, bias=True, ragged=True, spare=3),
        # the smallest scan, where the call's own time counts
        dict(name="scan tiny fp32", op="scan_fwd", lens="64", packed=False, H=2, K=16, dtype="fp32", gate="logits", ingate=True, norm=True, s0=False),
        # a serving batch of one layer: packed prompts
        dict(name="scan prompts", op="scan_fwd", lens="3001,1,517,0,1024,64,1300,2049", packed=True, H=32, K=128, dtype="bf16", gate="logits", ingate=True, norm=True, s0=True),
        # one very long row of few channels, decays as given
        dict(name="scan long", op="scan_fwd", lens="131072", packed=False, H=4, K=64, dtype="bf16", gate="log", ingate=False, norm=False, s0=False),
        # a training step of one layer, forward and gradients
        dict(name="scan training", op="scan_train", lens="4096,4096", packed=False, H=32, K=128, dtype="bf16", gate="logits", ingate=True, norm=True, s0=False),
        # decoding for a full batch, one token each
        dict(name="scan step", op="scan_step", B=64, S=1, H=96, K=128, dtype="bf16", gate="logits", ingate=True, norm=True, ragged=False, spare=0),
        # behind the heads of one layer's recurrence: norm and sigmoid gate
        dict(name="head norm", op="norm_fwd", tokens=8192, heads=96, D=128, dtype="bf16", gate="sigmoid", residual="none", after=True, before=False, scale=1.0, wide=False),
        # its gradients in a smaller layer, silu gate
        dict(name="head norm gradients", op="norm_bwd", tokens=4096, heads=32, D=128, dtype="bf16", gate="silu", residual="none", after=True, before=False, scale=1.0, wide=True),
        # between two blocks, decoding for one request: latency
        dict(name="block norm one", op="norm_fwd", tokens=1, heads=1, D=7168, dtype="bf16", gate="sigmoid", residual="bf16", after=True, before=True, scale=0.5, wide=False),
        # between two blocks, a training step's gradients, the residual stream in full precision
        dict(name="block norm gradients", op="norm_bwd", tokens=8192, heads=1, D=7168, dtype="bf16", gate="sigmoid", residual="fp32", after=True, before=True, scale=0.5, wide=False),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv_fwd", "conv_bwd", "conv_step", "scan_fwd", "scan_fwd", "scan_train", "scan_train", "scan_step", "norm_fwd", "norm_fwd", "norm_bwd", "norm_bwd"])
    dtype, odd = rng.choice(["fp32", "bf16", "bf16"]), rng.random() < 0.3
    if op.startswith("norm"):
        D = _log(rng, 1, 8192) if odd else 8 * _log(rng, 1, 1024)
        rows = _log(rng, 1, max(1, min(1 << 20, (40 << 20) // D)))
        heads = rng.choice([1, 1, 2, 16, 96])
        residual = rng.choice(["none", dtype, "fp32"])
        after = rng.random() < 0.7
        return dict(op=op, tokens=max(1, rows // heads), heads=heads, D=D, dtype=dtype, gate=rng.choice(["none", "sigmoid", "silu"]), residual=residual,
                    after=after, before=not after or residual != "none", scale=rng.choice([1.0, 0.5, 0.1]), wide=rng.random() < 0.3)
    H, K = (_log(rng, 1, 200), rng.choice([1, 3, 20, 33])) if odd else (_log(rng, 1, 96), rng.choice([8, 64, 128]))
    C = H * K
    if op.endswith("step"):
        S = rng.choice([1, 1, 2, 3, 5])
        case = dict(op=op, B=_log(rng, 1, 256 // S), S=S, ragged=rng.random() < 0.5, spare=rng.randint(0, 3))
    else:
        total = _log(rng, 1, max(1, min(1 << 17, (24 << 20) // C)))
        packed = rng.random() < 0.5
        if packed:
            n = rng.randint(2, 9)
            cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
            lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
        else:
            n = rng.choice([1, 1, 2, 3])
            lens = [max(1, total // n)] * n
        case = dict(op=op, lens=",".join(map(str, lens)), packed=packed, s0=rng.random() < 0.5)
    if op.startswith("conv"):
        case.update(D=C, W=rng.choice([2, 3, 4, 4]), dtype=dtype, silu=rng.random() < 0.7, bias=rng.random() < 0.5)
        return case if op.endswith("step") else dict(case, wide=rng.random() < 0.3)
    return dict(case, H=H, K=K, dtype=dtype, gate=rng.choice(["logits", "logits", "log"]), ingate=rng.random() < 0.6, norm=rng.random() < 0.6)


# --------------------------------------------------------------------------- the inputs

def _type(name):
    return torch.float32 if name == "fp32" else torch.bfloat16


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    t = _type(case["dtype"])

    def rows(*shape):  # activations; the wide ones are a slice of a projection that makes several at once
        if case.get("wide"):
            return rand(*shape[:-1], 2 * shape[-1] + 8).to(t)[..., 8 : 8 + shape[-1]]
        return rand(*shape).to(t)

    s = dict(case=case)
    if case["op"].startswith("norm"):
        shape = (case["tokens"], case["heads"], case["D"])
        s["y"] = (1.5 * rand(*shape)).to(t)
        s["gate"] = rows(*shape) if case["gate"] != "none" else None
        s["w_after"] = 1 + 0.2 * rand(case["D"]) if case["after"] else None
        s["w_before"] = 1 + 0.2 * rand(case["D"]) if case["before"] else None
        s["residual"] = (2 * rand(*shape)).to(_type(case["residual"])) if case["residual"] != "none" else None
        if case["op"] == "norm_bwd":
            # the stream that the forward left, and the gradients that come back: of the stream and of the next block's input
            s["h"] = (s["residual"] if s["residual"] is not None else s["y"]) + rand(*shape).to(t) if case["before"] else None
            ht = _type(case["residual"] if case["residual"] != "none" else case["dtype"])
            s["h"] = s["h"].to(ht) if s["h"] is not None else None
            s["residual"] = None
            s["d_h"] = rand(*shape).to(ht)
            s["d_n"] = rand(*shape).to(t) if case["before"] else None
        return s
    step = case["op"].endswith("step")
    if step:
        B, S = case["B"], case["S"]
        lead, P = (B, S), B * S + case["spare"]
        s["slots"] = torch.randperm(P, generator=gen, device="cuda")[: B * S].reshape(B, S).to(torch.int32)
        # how many of the last drafts were taken: the state to go on from
        s["start"] = torch.randint(0, S, (B,), generator=gen, device="cuda").to(torch.int32) if S > 1 else None
        s["lengths"] = torch.randint(1, S + 1, (B,), generator=gen, device="cuda").to(torch.int32) if case["ragged"] else None
    else:
        lens = [int(x) for x in case["lens"].split(",")]
        lead = (1, sum(lens)) if case["packed"] else (len(lens), lens[0])
        s["cu"] = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda") if case["packed"] else None
        P = len(lens)
    if case["op"].startswith("conv"):
        D, W = case["D"], case["W"]
        s["x"] = rows(*lead, D)
        s["weight"] = rand(D, W) * W ** -0.5
        s["bias"] = 0.2 * rand(D) if case["bias"] else None
        s["states" if step else "s0"] = rand(P, W - 1, D).to(t) if step or case["s0"] else None
        if step:
            s["out"] = torch.zeros(*lead, D, device="cuda", dtype=t)
        if case["op"] == "conv_bwd":
            s["d_out"], s["d_final"] = rand(*lead, D).to(t), rand(P, W - 1, D).to(t)
        return s
    H, K = case["H"], case["K"]
    s["x"] = rand(*lead, H, K).to(t)
    s["in_gate"] = rand(*lead, H, K).to(t) if case["ingate"] else None
    s["log_scale"] = s["bias"] = None
    if case["gate"] == "logits":  # channels that forget in a few tokens up to ones that keep for a thousand
        s["gate"] = rand(*lead, H, K).to(t)
        s["log_scale"], s["bias"] = 0.3 * rand(H), -6 + 6 * torch.rand(H, K, generator=gen, device="cuda")
    else:
        rate = torch.exp(math.log(1e-3) + math.log(1e3) * torch.rand(H, K, generator=gen, device="cuda"))
        s["gate"] = -torch.nn.functional.softplus(rand(*lead, H, K)) * rate
    s["states" if step else "s0"] = rand(P, H, K) if step or case["s0"] else None
    if step:
        s["out"] = torch.zeros(*lead, H, K, device="cuda", dtype=t)
    if case["op"] == "scan_train":
        s["d_out"], s["d_final"] = rand(*lead, H, K).to(t), rand(P, H, K)
    return s


def work(case):
    e = 4 if case["dtype"] == "fp32" else 2
    if case["op"].startswith("norm"):
        n = case["tokens"] * case["heads"] * case["D"]
        r = 0 if case["residual"] == "none" else 4 if case["residual"] == "fp32" else e
        gate = 0 if case["gate"] == "none" else e
        if case["op"] == "norm_fwd":
            return {"bytes": n * (e + gate + r + (r or e) + (e if case["before"] else 0)) + 8.0 * case["D"], "flops": 16.0 * n}
        # y, the gate, d_h and with a norm before h and d_n; their gradients
        return {"bytes": n * (2 * e + 2 * gate + (r or e) + (2 * (r or e) + e if case["before"] else 0)) + 16.0 * case["D"], "flops": 40.0 * n}
    conv = case["op"].startswith("conv")
    C = case["D"] if conv else case["H"] * case["K"]
    if case["op"].endswith("step"):  # a state read for each request and one written for each token
        n = case["B"] * case["S"] * ((case["S"] + 1) / (2 * case["S"]) if case["ragged"] else 1)
        state = (case["W"] - 1) * e if conv else 4
        gates = 0 if conv else (e if case["gate"] == "logits" else 4) + (e if case["ingate"] else 0)
        return {"bytes": C * (state * (case["B"] + n) + n * (2 * e + gates)), "flops": 20.0 * n * C}
    lens = [int(x) for x in case["lens"].split(",")]
    n = sum(lens) * C
    if conv:
        states = (2 if case["s0"] else 1) * len(lens) * (case["W"] - 1) * C * e
        if case["op"] == "conv_fwd":
            return {"bytes": 2.0 * e * n + states + 4 * C * (case["W"] + 1), "flops": n * (2.0 * case["W"] + 6)}
        return {"bytes": 3.0 * e * n + states + 8 * C * (case["W"] + 1), "flops": n * (6.0 * case["W"] + 12)}
    states = (2 if case["s0"] else 1) * len(lens) * C * 4.0
    ins = e + (e if case["gate"] == "logits" else 4) + (e if case["ingate"] else 0)
    if case["op"] == "scan_fwd":
        return {"bytes": n * (ins + e) + states, "flops": 25.0 * n}
    return {"bytes": n * (2 * ins + 2 * e) + 2 * states, "flops": 75.0 * n}


# --------------------------------------------------------------------------- the operators

def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if own:
        import gated_delta_rule_31_amd as kda
        if op == "conv_fwd":
            return kda.short_conv_fwd(s["x"], s["weight"], bias=s["bias"], initial_state=s["s0"], cu_seqlens=s["cu"], silu=case["silu"])
        if op == "conv_bwd":
            return kda.short_conv_bwd(s["x"], s["weight"], s["d_out"], bias=s["bias"], initial_state=s["s0"], d_final_state=s["d_final"],
                                      cu_seqlens=s["cu"], silu=case["silu"])
        if op == "conv_step":
            out = kda.short_conv_step(s["x"], s["weight"], s["states"], bias=s["bias"], slots=s["slots"], start=s["start"], lengths=s["lengths"],
                                      silu=case["silu"], out=s["out"])
            return out, s["states"]
        gates = dict(log_scale=s.get("log_scale"), bias=s.get("bias"), in_gate=s.get("in_gate"), normalize=case.get("norm"), lower_bound=LOWER)
        if op == "scan_fwd":
            return kda.glr_fwd(s["x"], s["gate"], initial_state=s["s0"], cu_seqlens=s["cu"], **gates)
        if op == "scan_train":
            out, final, kept = kda.glr_fwd(s["x"], s["gate"], initial_state=s["s0"], cu_seqlens=s["cu"], keep=True, **gates)
            return out, final, kda.glr_bwd(s["x"], s["gate"], s["d_out"], initial_state=s["s0"], d_final_state=s["d_final"], cu_seqlens=s["cu"],
                                           kept=kept, **gates)
        if op == "scan_step":
            out = kda.glr_step(s["x"], s["gate"], s["states"], slots=s["slots"], start=s["start"], lengths=s["lengths"], out=s["out"], **gates)
            return out, s["states"]
        parts = dict(gate=s["gate"], weight_after=s["w_after"], weight_before=s["w_before"], norm_after=case["after"], norm_before=case["before"],
                     scale=case["scale"], eps=EPS, silu=case["gate"] == "silu")
        if op == "norm_fwd":
            return kda.block_norm_fwd(s["y"], residual=s["residual"], **parts)
        return kda.block_norm_bwd(s["y"], s["d_h"], d_n=s["d_n"], h=s["h"], **parts)
    if op == "norm_fwd":
        return _plain_norm(s)
    if op == "norm_bwd":
        return _plain_norm_bwd(s)
    if op == "conv_step":
        return _plain_step(s, _conv_token)
    if op == "scan_step":
        return _plain_step(s, _scan_token)
    if op == "conv_fwd":
        return _plain_conv(s)
    if op == "conv_bwd":
        return _plain_conv_bwd(s)
    f = _plain_scan(s)
    if op == "scan_fwd":
        return f["out"].to(s["x"].dtype).reshape(s["x"].shape), f["final"]
    return f["out"].to(s["x"].dtype).reshape(s["x"].shape), f["final"], _plain_scan_bwd(s, f)


def _places(s, lead):
    """Of every row of a batch: its sequence, its place in it and the sequence's length; and the sequences' bounds."""
    B, T = lead
    device = s["x"].device
    cu = s["cu"].long() if s["cu"] is not None else torch.arange(B + 1, device=device) * T
    at = torch.arange(B * T, device=device)
    seq = torch.searchsorted(cu, at, right=True) - 1
    return seq, at - cu[seq], (cu[1:] - cu[:-1])[seq], cu


def _silu_slope(x):
    g = torch.sigmoid(x)
    return g * (1 + x * (1 - g))


def _taps(s, W):
    """x_{t-j} for j = 0 .. W-1 in 32 bits, from the kept rows (or zeros) where that is before the sequence."""
    x = s["x"].float().reshape(-1, s["x"].shape[-1])
    seq, pos, size, cu = _places(s, s["x"].shape[:2])
    kept = s["s0"].float() if s["s0"] is not None else torch.zeros(len(cu) - 1, W - 1, x.shape[1], device=x.device)
    at = torch.arange(len(x), device=x.device)
    taps = [torch.where((pos >= j)[:, None], x[(at - j).clamp_min(0)], kept[seq, (W - 1 + pos - j).clamp(0, W - 2)]) for j in range(W)]
    return taps, kept, seq, pos, size, cu


def _plain_conv(s):
    W = s["weight"].shape[1]
    taps, kept, seq, pos, size, cu = _taps(s, W)
    pre = sum(taps[j] * s["weight"][:, W - 1 - j] for j in range(W))
    pre = pre + s["bias"] if s["bias"] is not None else pre
    out = pre * torch.sigmoid(pre) if s["case"]["silu"] else pre
    x = s["x"].reshape(-1, s["x"].shape[-1])
    at = (cu[1:] - cu[:-1])[:, None] - (W - 1) + torch.arange(W - 1, device=x.device)  # places of the last rows
    final = torch.where((at >= 0)[..., None], x[(cu[:-1, None] + at).clamp(0, len(x) - 1)].float(), kept.gather(1, (at + W - 1).clamp(0, W - 2)[..., None].expand(-1, -1, x.shape[1])))
    return out.to(x.dtype).reshape(s["x"].shape), final.to(x.dtype)


def _plain_conv_bwd(s):
    w, W, D = s["weight"], s["weight"].shape[1], s["x"].shape[-1]
    taps, kept, seq, pos, size, cu = _taps(s, W)
    d = s["d_out"].float().reshape(-1, D)
    if s["case"]["silu"]:
        pre = sum(taps[j] * w[:, W - 1 - j] for j in range(W))
        d = d * _silu_slope(pre + s["bias"] if s["bias"] is not None else pre)
    at = torch.arange(len(d), device=d.device)
    dx = sum(torch.where((pos + j < size)[:, None], d[(at + j).clamp_max(len(d) - 1)], 0) * w[:, W - 1 - j] for j in range(W))
    dw = torch.stack([(d * taps[W - 1 - j]).sum(0, dtype=torch.float64) for j in range(W)], 1).float()
    db = d.sum(0, dtype=torch.float64).float() if s["bias"] is not None else None
    # kept row r is read by the places p <= r, through tap W - 1 + p - r; what was handed on goes back to the rows it was made of
    ds, n = torch.zeros_like(kept), cu[1:] - cu[:-1]
    for r in range(W - 1):
        for p in range(r + 1):
            ds[:, r] += torch.where((p < n)[:, None], d[(cu[:-1] + p).clamp_max(len(d) - 1)], 0) * w[:, r - p]
    for r in range(W - 1):
        place, given = n - (W - 1) + r, s["d_final"][:, r].float()
        dx = dx.index_add(0, (cu[:-1] + place).clamp(0, len(d) - 1), given * (place >= 0)[:, None])
        ds = ds.scatter_add(1, (n + r).clamp_max(W - 2)[:, None, None].expand(-1, 1, D), (given * (place < 0)[:, None])[:, None])
    t = s["x"].dtype
    return dx.to(t).reshape(s["x"].shape), dw, db, ds.to(t)


def _gates(s, flat=True):
    """Log decays and what multiplies x, in 32 bits."""
    g = s["gate"].float()
    if s["log_scale"] is not None:
        g = LOWER * torch.sigmoid(torch.exp(s["log_scale"])[:, None] * (g + s["bias"]))
    f = torch.sqrt(-torch.expm1(2 * g)) if s["case"]["norm"] else torch.ones_like(g)
    i = torch.sigmoid(s["in_gate"].float()) if s["in_gate"] is not None else torch.ones_like(g)
    return [y.reshape(-1, y.shape[-2] * y.shape[-1]) if flat else y for y in (g, f, i)]


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t for all rows, by spans that double."""
    n = 1
    while n < len(a):
        b = torch.cat([b[:n], b[n:] + a[n:] * b[:-n]])
        a = torch.cat([a[:n], a[n:] * a[:-n]])
        n *= 2
    return b


def _plain_scan(s):
    C = s["x"].shape[2] * s["x"].shape[3]
    g, f, i = _gates(s)
    x, a = s["x"].float().reshape(-1, C), torch.exp(g)
    seq, pos, size, cu = _places(s, s["x"].shape[:2])
    N = len(cu) - 1
    s0 = s["s0"].reshape(N, C) if s["s0"] is not None else torch.zeros(N, C, device=x.device)
    first = (pos == 0)[:, None]
    h = _scan(torch.where(first, 0, a), torch.where(first, a * s0[seq], 0) + f * i * x)
    final = torch.where((cu[1:] > cu[:-1])[:, None], h[(cu[1:] - 1).clamp_min(0)], s0)
    return dict(out=h, final=final.reshape(N, *s["x"].shape[2:]), g=g, f=f, i=i, a=a, x=x, s0=s0, seq=seq, pos=pos, size=size, cu=cu)


def _plain_scan_bwd(s, f):
    shape = s["x"].shape
    C, t = shape[2] * shape[3], s["x"].dtype
    a, x, h, cu, first, last = f["a"], f["x"], f["out"], f["cu"], (f["pos"] == 0)[:, None], (f["pos"] == f["size"] - 1)[:, None]
    d_final = s["d_final"].reshape(-1, C)
    d = s["d_out"].float().reshape(-1, C) + torch.where(last, d_final[f["seq"]], 0)
    after = torch.where(last, 0, torch.cat([a[1:], a[:1]]))  # the decay between a row and the next
    d = _scan(after.flip(0), d.flip(0)).flip(0)
    before = torch.where(first, f["s0"][f["seq"]], torch.cat([h[:1], h[:-1]]))
    dg = d * before * a
    dx, di = d * f["f"] * f["i"], d * f["f"] * x * f["i"] * (1 - f["i"])
    if s["case"]["norm"]:  # d sqrt(1 - e^{2g}) / dg = -e^{2g} / sqrt(1 - e^{2g})
        dg = dg - d * f["i"] * x * a * a / f["f"]
    ds0 = torch.where((cu[1:] > cu[:-1])[:, None], (a * d)[cu[:-1].clamp_max(len(a) - 1)], d_final)
    dA = db = None
    if s["log_scale"] is not None:
        scale = torch.exp(s["log_scale"]).repeat_interleave(shape[3])
        p = f["g"] / LOWER
        u = scale * (s["gate"].float().reshape(-1, C) + s["bias"].reshape(-1))
        du = dg * LOWER * p * torch.sigmoid(-u)
        dA = (u * du).sum(0, dtype=torch.float64).reshape(shape[2:]).sum(1).float()
        dg = scale * du
        db = dg.sum(0, dtype=torch.float64).reshape(shape[2:]).float()
    return (dx.to(t).reshape(shape), dg.to(s["gate"].dtype).reshape(shape), di.to(t).reshape(shape) if s["in_gate"] is not None else None, dA, db,
            ds0.reshape(-1, *shape[2:]))


def _conv_token(s, state, x, t):
    """Kept rows [B, W - 1, D] and one token of each request -> (output, kept rows)."""
    rows = torch.cat([state, x[:, None]], 1)
    pre = (rows * s["weight"].t()).sum(1)
    pre = pre + s["bias"] if s["bias"] is not None else pre
    return pre * torch.sigmoid(pre) if s["case"]["silu"] else pre, rows[:, 1:]


def _scan_token(s, state, x, t):
    g, f, i = (y[:, t] for y in _gates(s, False))
    h = torch.exp(g) * state + f * i * x
    return h, h


def _plain_step(s, token):
    """One token after another; the state after each goes to its slot."""
    x, states, out, slots = s["x"].float(), s["states"], s["out"], s["slots"].long()
    B, S = slots.shape
    rows = torch.arange(B, device=x.device)
    start = s["start"].long() if s["start"] is not None else torch.zeros_like(rows)
    lengths = s["lengths"] if s["lengths"] is not None else torch.full_like(rows, S)
    kept = states[slots[rows, start]].float()
    for t in range(S):
        there = (t < lengths).reshape(-1, *[1] * (x.dim() - 2))
        y, new = token(s, kept, x[:, t], t)
        kept = torch.where(there.reshape(-1, *[1] * (kept.dim() - 1)), new, kept)
        states[slots[:, t]] = torch.where(there.reshape(-1, *[1] * (kept.dim() - 1)), kept.to(states.dtype), states[slots[:, t]])
        out[:, t] = torch.where(there, y.to(out.dtype), out[:, t])
    return out, states


def _act(s):
    z = s["gate"].float()
    return z, torch.sigmoid(z)


def _rms(x):
    return torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)


def _plain_norm(s):
    case, y = s["case"], s["y"].float()
    p = y * _rms(y) * s["w_after"] if case["after"] else y
    if s["gate"] is not None:
        z, g = _act(s)
        p = p * (z * g if case["gate"] == "silu" else g)
    h = case["scale"] * p
    h = s["residual"].float() + h if s["residual"] is not None else h
    n = (h * _rms(h) * s["w_before"]).to(s["y"].dtype) if case["before"] else None
    return h.to(s["residual"].dtype if s["residual"] is not None else s["y"].dtype), n


def _plain_norm_bwd(s):
    case, y, dh, D = s["case"], s["y"].float(), s["d_h"].float(), s["y"].shape[-1]
    dwa = dwb = dz = None
    total = lambda x: x.reshape(-1, D).sum(0, dtype=torch.float64).float()  # noqa: E731
    if case["before"]:
        h, dn = s["h"].float(), s["d_n"].float()
        r = _rms(h)
        u = h * r
        dwb = total(dn * u)
        du = dn * s["w_before"]
        dh = dh + r * (du - u * (du * u).mean(-1, keepdim=True))
    r = _rms(y) if case["after"] else 1.0
    v = y * r
    p = v * s["w_after"] if case["after"] else v
    dp = case["scale"] * dh
    if s["gate"] is not None:
        z, g = _act(s)
        act, slope = (z * g, g * (1 + z * (1 - g))) if case["gate"] == "silu" else (g, g * (1 - g))
        dz = (dp * p * slope).to(s["gate"].dtype)
        dp = dp * act
    dy = dp
    if case["after"]:
        dwa = total(dp * v)
        dv = dp * s["w_after"]
        dy = r * (dv - v * (dv * v).mean(-1, keepdim=True))
    return dy.to(s["y"].dtype), dz, dh.to(s["d_h"].dtype), dwa, dwb


# --------------------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    wide = lambda n: s[n].double() if s.get(n) is not None else None  # noqa: E731
    if case["op"].startswith("norm"):
        # by automatic differentiation of the definition, a few rows at a time; the stream that the norm before
        # reads is the one that was stored
        D, rows = case["D"], case["tokens"] * case["heads"]
        flat = {n: (s[n].reshape(rows, D) if s.get(n) is not None else None) for n in ("y", "gate", "residual", "h", "d_h", "d_n")}
        wa, wb = wide("w_after"), wide("w_before")
        back = case["op"] == "norm_bwd"
        for w in (wa, wb):
            if w is not None and back:
                w.requires_grad_()
        norm = lambda x, w: w * x / ((x ** 2).sum(-1, keepdim=True) / D + EPS).sqrt()  # noqa: E731
        parts = []
        step = max(1, (1 << 24) // D)
        for at in range(0, rows, step):
            y, z, res, h, d_h, d_n = (flat[n][at : at + step].double() if flat[n] is not None else None for n in ("y", "gate", "residual", "h", "d_h", "d_n"))
            leaves = [x.requires_grad_() for x in (y, z, h) if x is not None] if back else []
            p = norm(y, wa) if case["after"] else y
            if z is not None:
                p = p / (1 + torch.exp(-z)) * (z if case["gate"] == "silu" else 1)
            p = case["scale"] * p
            if not back:
                p = p if res is None else res + p
                parts.append((p, norm(p, wb) if case["before"] else None))
                continue
            through = None
            if case["before"]:
                (norm(h, wb) * d_n).sum().backward()
                through = h.grad
            d_h = d_h if through is None else d_h + through
            (p * d_h).sum().backward()
            parts.append((y.grad, z.grad if z is not None else None, d_h))
        shape = s["y"].shape
        outs = [None if parts[0][k] is None else torch.cat([q[k] for q in parts]).reshape(shape) for k in range(len(parts[0]))]
        return tuple(outs) if not back else tuple(outs) + tuple(None if w is None else w.grad for w in (wa, wb))
    conv = case["op"].startswith("conv")
    sig = lambda x: 1 / (1 + torch.exp(-x))  # noqa: E731

    def token(x, kept, at):
        """One row of a sequence (or one token of all requests, at `at`)."""
        if conv:
            rows = torch.cat([kept, x.unsqueeze(-2)], -2)
            pre = (rows * wide("weight").T).sum(-2) + (wide("bias") if case["bias"] else 0)
            return (pre * sig(pre) if case["silu"] else pre), rows[..., 1:, :]
        z = s["gate"][at].double()
        g = z if case["gate"] == "log" else LOWER * sig(wide("log_scale").exp()[:, None] * (z + wide("bias")))
        h = g.exp() * kept + ((1 - (2 * g).exp()).sqrt() if case["norm"] else 1) * (sig(s["in_gate"][at].double()) if case["ingate"] else 1) * x
        return h, h

    if case["op"].endswith("step"):
        states, out = wide("states"), wide("out")
        slots = s["slots"].tolist()
        start = s["start"].tolist() if s["start"] is not None else [0] * case["B"]
        lengths = s["lengths"].tolist() if s["lengths"] is not None else [case["S"]] * case["B"]
        for b in range(case["B"]):
            kept = states[slots[b][start[b]]].clone()
            for t in range(lengths[b]):
                out[b, t], kept = token(s["x"][b, t].double(), kept, (b, t))
                states[slots[b][t]] = kept.to(s["states"].dtype).double() if conv else kept
        return out, states
    lens = [int(x) for x in case["lens"].split(",")]
    N, C = len(lens), s["x"].shape[2:].numel()
    x = wide("x").reshape(-1, C)
    bounds = [(sum(lens[:i]), sum(lens[: i + 1])) for i in range(N)]
    if conv:
        W = case["W"]
        w, b = wide("weight"), wide("bias")
        s0 = wide("s0") if case["s0"] else torch.zeros(N, W - 1, C, device="cuda", dtype=torch.float64)
        outs, finals, grads = [], [], []
        dw, db = torch.zeros_like(w), torch.zeros_like(b) if b is not None else None
        for i, (lo, hi) in enumerate(bounds):
            rows = torch.cat([s0[i], x[lo:hi]])
            if hi == lo:
                outs.append(x[lo:hi])
                finals.append(rows)
                grads.append((x[lo:hi], wide("d_final")[i] if case["op"] == "conv_bwd" else None))
                continue
            pre = rows.unfold(0, W, 1) @ torch.eye(W, device="cuda", dtype=torch.float64)
            pre = (pre * w).sum(-1) + (b if b is not None else 0)
            outs.append(pre * sig(pre) if case["silu"] else pre)
            finals.append(rows[hi - lo :])
            if case["op"] == "conv_bwd":
                d = wide("d_out").reshape(-1, C)[lo:hi]
                d = d * (sig(pre) + pre * sig(pre) * sig(-pre)) if case["silu"] else d
                back = torch.zeros_like(rows)
                for j in range(W):
                    back[j : j + hi - lo] += d * w[:, j]
                    dw[:, j] += (d * rows[j : j + hi - lo]).sum(0)
                if db is not None:
                    db += d.sum(0)
                back[hi - lo :] += wide("d_final")[i]
                grads.append((back[W - 1 :], back[: W - 1]))
        if case["op"] == "conv_fwd":
            return torch.cat(outs).reshape(s["x"].shape), torch.stack(finals)
        return torch.cat([q[0] for q in grads]).reshape(s["x"].shape), dw, db, torch.stack([q[1] for q in grads])
    # the scan, token by token
    z = wide("gate").reshape(-1, C)
    if case["gate"] == "logits":
        A = wide("log_scale").repeat_interleave(case["K"])
        u = A.exp() * (z + wide("bias").reshape(-1))
        p = sig(u)
        z = LOWER * p
    a = z.exp()
    f = (1 - (2 * z).exp()).sqrt() if case["norm"] else torch.ones_like(z)
    i = sig(wide("in_gate").reshape(-1, C)) if case["ingate"] else torch.ones_like(z)
    b = f * i * x
    s0 = wide("s0").reshape(N, C) if case["s0"] else torch.zeros(N, C, device="cuda", dtype=torch.float64)
    h, final = torch.empty_like(x), s0.clone()
    for n, (lo, hi) in enumerate(bounds):
        for t in range(lo, hi):
            torch.addcmul(b[t], a[t], h[t - 1] if t > lo else s0[n], out=h[t])
        if hi > lo:
            final[n] = h[hi - 1]
    shape = s["x"].shape
    out = h.reshape(shape), final.reshape(N, *shape[2:])
    if case["op"] == "scan_fwd":
        return out
    d, ds0, d_final = wide("d_out").reshape(-1, C).clone(), torch.empty_like(s0), wide("d_final").reshape(N, C)
    before = torch.empty_like(h)
    for n, (lo, hi) in enumerate(bounds):
        for t in reversed(range(lo, hi)):
            if t == hi - 1:
                d[t] += d_final[n]
            else:
                d[t].addcmul_(a[t + 1], d[t + 1])
        before[lo + 1 : hi] = h[lo : hi - 1] if hi > lo else h[:0]
        if hi > lo:
            before[lo] = s0[n]
        ds0[n] = a[lo] * d[lo] if hi > lo else d_final[n]
    dg = d * (before * a - (i * x * a * a / f if case["norm"] else 0))
    dx, di = d * f * i, d * f * x * i * (1 - i)
    dA = db = None
    if case["gate"] == "logits":
        du = dg * LOWER * p * (1 - p)
        dA, dg = (u * du).sum(0).reshape(shape[2:]).sum(1), A.exp() * du
        db = dg.sum(0).reshape(shape[2:])
    return out + ((dx.reshape(shape), dg.reshape(shape), di.reshape(shape) if case["ingate"] else None, dA, db, ds0.reshape(N, *shape[2:])),)
