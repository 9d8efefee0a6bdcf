"""What stands around the recurrence in a layer, in the forms in which it is trained and served: a whole
block against its 64-bit form, decoding with drafts through one table of slots, captured and
replayed calls, several streams, rows and pools past 32-bit offsets."""
import pytest
import torch

import gated_delta_rule_31_amd as kda
from tests import layer_reference as ref
from tests.layer_reference import f64
from tests.test_gpu_layer import close, conv_case, gen, gpu, norm_case, offsets, scan_case

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


# --------------------------------------------------------------------------- together

def _block(op, y, x, w1, w2, conv_w, conv_b, log_scale, bias, norm_a, norm_b, heads, width):
    """norm between blocks -> projection -> convolution -> recurrence -> gated head norm -> projection -> norm between blocks"""
    h, n = op.block_norm(y, residual=x, weight_after=norm_a, weight_before=norm_b, scale=0.5)
    u = n @ w1  # recurrence's input, its gate's logits, its input gate and the output gate side by side
    C = heads * width
    v, _ = op.short_conv(u[..., :C], conv_w, conv_b)
    part = lambda k: u[..., k * C : (k + 1) * C].unflatten(-1, (heads, width))  # noqa: E731
    r, final = op.scan(v.unflatten(-1, (heads, width)), part(1), log_scale, bias, part(2))
    o = op.gated_norm(r, part(3))
    h, n = op.block_norm(o.flatten(-2) @ w2, residual=h, weight_after=norm_b, weight_before=norm_a, scale=0.5, gate=n)
    return h, n, final


class _Ours:
    def __init__(self, lens):
        self.cu = gpu(offsets(lens))

    def block_norm(self, y, **kw):
        return kda.block_norm(y, silu=True, **kw)

    def gated_norm(self, y, gate):
        return kda.gated_norm(y, gate)

    def short_conv(self, x, w, b):
        return kda.short_conv(x, w, b, cu_seqlens=self.cu)

    def scan(self, x, z, a, b, i):
        return kda.gated_linear_recurrence(x, z, a, b, i, cu_seqlens=self.cu)


class _Plain:
    def __init__(self, lens):
        self.lens = lens

    def block_norm(self, y, residual, weight_after, weight_before, scale, gate=None):
        return ref.block_norm(y, gate, residual, weight_after, weight_before, True, True, scale, 1e-6, True)

    def gated_norm(self, y, gate):
        return ref.block_norm(y, gate, None, None, None, True, False, 1.0, 1e-6, False)[0]

    def short_conv(self, x, w, b):
        return ref.conv(x, w, b, None, self.lens, True)

    def scan(self, x, z, a, b, i):
        return ref.scan(x, z, a, b, i, None, self.lens, True)


@pytest.mark.parametrize("lens", [[70, 0, 33, 1], [200]])
def test_recurrent_block_trains(lens):
    """A block's outputs and all its gradients.  Each of its seven stages is off by at most 6 x 1024 roundings of 2^-24 in an
    element, 3.7e-4 of the rms, and as these are independent by a tenth of that in the 2-norm: 7 x 3.7e-5 = 2.6e-4."""
    D, H, K, T = 48, 2, 24, sum(lens)
    r = gen(40)
    C = H * K
    data = [r(1, T, D), 2 * r(1, T, D), r(D, 4 * C) * D ** -0.5, r(C, D) * C ** -0.5, r(C, 4) * 0.5, 0.2 * r(C), 0.2 * r(H), r(H, K) - 1, 1 + 0.2 * r(D), 1 + 0.2 * r(D)]
    gh, gn, gf = r(1, T, D), r(1, T, D), r(len(lens), H, K)
    mine, plain = [gpu(t).requires_grad_() for t in data], [f64(t).requires_grad_() for t in data]
    got, want = _block(_Ours(lens), *mine, H, K), _block(_Plain(lens), *plain, H, K)
    for u, v, name in zip(got, want, ("h", "n", "final")):
        assert float((f64(u) - v.detach()).norm() / v.detach().norm()) <= 2.6e-4, name
    grads = torch.autograd.grad(sum((u * gpu(g)).sum() for u, g in zip(got, (gh, gn, gf))), mine)
    refs = torch.autograd.grad(sum((u * f64(g)).sum() for u, g in zip(want, (gh, gn, gf))), plain)
    for k, (u, v) in enumerate(zip(grads, refs)):
        assert float((f64(u) - v).norm() / v.norm()) <= 2.6e-4, k


def test_layer_decodes_with_drafts():
    """Convolution, gated delta rule and linear recurrence go by one table of slots through rounds of drafts, and give what
    their prefills give.  Float32: 512 roundings (test_gpu_layer) for the linear parts, 1e-4 for the delta rule's."""
    B, T, S, H, K = 4, 17, 3, 2, 16
    r = gen(41)
    C = H * K
    x, w, g, beta, z = r(B, T, C), r(C, 4) / 2, -0.5 * r(B, T, H).abs(), torch.sigmoid(r(B, T, H)), r(B, T, H, K)
    ls, b = 0.1 * r(H), r(H, K)
    x, w, g, beta, z, ls, b = map(gpu, (x, w, g, beta, z, ls, b))
    unit = lambda t: t / t.norm(dim=-1, keepdim=True)  # noqa: E731
    conv = kda.short_conv_fwd(x, w)[0].unflatten(-1, (H, K))
    q = unit(conv)
    want = kda.gdr_chunk_fwd(q, q, conv, g, beta)[0], kda.glr_fwd(conv, z, ls, b)[0]
    pool = B * S
    slots = torch.randperm(pool, generator=torch.Generator().manual_seed(3)).reshape(B, S).int().cuda()
    rows, deltas, states = (torch.zeros(pool, *s, device="cuda") for s in ((3, C), (H, K, K), (H, K)))
    at, start = [0] * B, torch.zeros(B, dtype=torch.int32, device="cuda")
    while min(at) < T:
        n = [min(S, T - t) for t in at]
        cut = lambda t: torch.stack([torch.cat([t[i, a : a + k], t.new_zeros(S - k, *t.shape[2:])]) for i, (a, k) in enumerate(zip(at, n))])  # noqa: E731
        kw = dict(slots=slots, start=start, lengths=torch.tensor(n, dtype=torch.int32, device="cuda"))
        c = kda.short_conv_step(cut(x), w, rows, **kw).unflatten(-1, (H, K))
        u = unit(c.where(c != 0, torch.full_like(c, 1e-20)))
        outs = kda.gdr_recurrent_step(u, u, c, cut(g), cut(beta), deltas, **kw), kda.glr_step(c, cut(z), states, ls, b, **kw)
        for i in range(B):
            if n[i]:
                close(outs[0][i, : n[i]], want[0][i, at[i] : at[i] + n[i]], 1700)
                close(outs[1][i, : n[i]], want[1][i, at[i] : at[i] + n[i]], 512)
                took = min(n[i], 1 + (at[i] + i) % S)
                start[i] = took - 1
                at[i] += took


# --------------------------------------------------------------------------- captured calls, streams

def _calls():
    """name -> (inputs, call of them that gives a list of tensors)"""
    lens = [70, 0, 130, 1]
    cu = gpu(offsets(lens))
    x, w, b, s = map(gpu, conv_case(lens, True, 40, 4, BF, True, True, 50))
    d = gpu(gen(51)(*x.shape).to(BF))
    X, z, ls, bi, i, s0 = map(gpu, scan_case(lens, True, 3, 24, BF, True, True, True, 52))
    D = gpu(gen(53)(*X.shape).to(BF))
    y, g, res, wa, wb = map(gpu, norm_case((50, 2, 136), BF, F32, True, True, True, 54))
    dh, dn = gpu(gen(55)(*y.shape)), gpu(gen(56)(*y.shape).to(BF))
    flat = lambda t: [u for u in t if u is not None]  # noqa: E731

    def scan(X, z, i, s0, D):
        out, fin, kept = kda.glr_fwd(X, z, ls, bi, i, initial_state=s0, cu_seqlens=cu, keep=True)
        return flat([out[:, : sum(lens)], fin] + list(kda.glr_bwd(X, z, D, ls, bi, i, initial_state=s0, cu_seqlens=cu, kept=kept)))

    def steps(x, X, z, i):
        rows, states = torch.zeros(70, 3, 40, dtype=BF, device="cuda"), torch.zeros(70, 3, 24, device="cuda")
        return [kda.short_conv_step(x[:, :70].transpose(0, 1).contiguous(), w, rows, b), rows, kda.glr_step(*(t[:, :70].transpose(0, 1).contiguous() for t in (X, z)), states,
                                                                                                       ls, bi, i[:, :70].transpose(0, 1).contiguous()), states]
    return {"conv": ([x, s, d], lambda x, s, d: flat(kda.short_conv_fwd(x, w, b, s, cu_seqlens=cu) + kda.short_conv_bwd(x, w, d, b, s, cu_seqlens=cu))),
            "scan": ([X, z, i, s0, D], scan), "steps": ([x, X, z, i], steps),
            "norm": ([y, g, res, dh, dn], lambda y, g, res, dh, dn: flat(kda.block_norm_fwd(y, g, res, wa, wb) + kda.block_norm_bwd(y, dh, dn, res, g, wa, wb)))}


@pytest.mark.parametrize("name", ["conv", "scan", "steps", "norm"])
def test_captured(name):
    """A captured call, replayed with other inputs between the program's own work, gives the eager call's bits every time."""
    inputs, call = _calls()[name]
    static = [t.clone() for t in inputs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(*static)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = call(*static)
    for k in range(4):
        new = [t * (1 + 0.25 * k) if t.is_floating_point() else t for t in inputs]
        for a, b in zip(static, new):
            a.copy_(b)
        want = call(*new)
        graph.replay()
        torch.cuda.synchronize()
        for u, v in zip(outs, want):
            assert torch.equal(u, v), k


def test_two_graphs_share_a_workspace():
    """Captured calls that share a caller's workspace, replayed one after the other, give the eager calls' bits."""
    lens, H, K = [300], 2, 16
    x, z, ls, b, i, s = map(gpu, scan_case(lens, False, H, K, F32, True, True, False, 57))
    x2 = x.flip(1).contiguous()
    d = gpu(gen(58)(*x.shape))
    ws = torch.empty(max(kda.glr_fwd_workspace_size(1, 300, H, K), kda.glr_bwd_workspace_size(1, 300, H, K, True, False)), dtype=torch.uint8, device="cuda")
    calls = [lambda: kda.glr_fwd(x, z, ls, b, i, workspace=ws), lambda: kda.glr_bwd(x2, z, d, ls, b, i, workspace=ws)]
    want = [[t.clone() for t in c() if t is not None] for c in calls]
    graphs, outs = [], []
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append([t for t in c() if t is not None])
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
        ws.fill_(255)  # the program's own use of it
        torch.cuda.synchronize()
        for got, ref_ in zip(outs, want):
            for u, v in zip(got, ref_):
                assert torch.equal(u, v)


def test_streams():
    """All calls at once on streams of their own, several times over, give what each gives alone."""
    calls = _calls()
    want = {n: call(*inputs) for n, (inputs, call) in calls.items()}
    torch.cuda.synchronize()
    streams = {n: torch.cuda.Stream() for n in calls}
    got = {n: [] for n in calls}
    for _ in range(3):
        for n, (inputs, call) in calls.items():
            with torch.cuda.stream(streams[n]):
                got[n].append(call(*inputs))
    torch.cuda.synchronize()
    for n in calls:
        for outs in got[n]:
            for u, v in zip(outs, want[n]):
                assert torch.equal(u, v), n


# --------------------------------------------------------------------------- past 32-bit offsets

def _far(rows, width, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(1, rows, width, generator=g, device="cuda", dtype=dtype)


def test_conv_past_32_bit_offsets():
    """The last rows of 2.4 x 10^9 numbers, and a pool of 2.3 x 10^9, are those of a small call."""
    T, D = 300_000, 8192
    x, w = _far(T, D, BF, 60), gpu(gen(61)(D, 4) / 2)
    tail = x[:, -100:].contiguous()
    out, fin = kda.short_conv_fwd(x, w)
    want, want_fin = kda.short_conv_fwd(tail, w, initial_state=x[:, -103:-100].contiguous())
    assert torch.equal(out[:, -100:], want) and torch.equal(fin, want_fin)
    dx, _, _, _ = kda.short_conv_bwd(x, w, out)
    ref_ = kda.short_conv_bwd(tail, w, want, initial_state=x[:, -103:-100].contiguous())[0]
    assert torch.equal(dx[:, -100:], ref_)
    del out, dx
    pool = torch.zeros(95_000, 3, D, dtype=BF, device="cuda")
    slots = torch.tensor([[94_999], [0], [90_000]], dtype=torch.int32, device="cuda")
    small = torch.zeros(3, 3, D, dtype=BF, device="cuda")
    for t in range(2):
        a = kda.short_conv_step(tail[:, 3 * t : 3 * t + 3].transpose(0, 1).contiguous(), w, pool, slots=slots)
        assert torch.equal(a, kda.short_conv_step(tail[:, 3 * t : 3 * t + 3].transpose(0, 1).contiguous(), w, small))
    assert torch.equal(pool[slots[:, 0].long()], small)


def test_scan_past_32_bit_offsets():
    T, H, K = 300_000, 64, 128
    x = _far(T, H * K, BF, 62).unflatten(-1, (H, K))
    ls = torch.zeros(H, device="cuda")
    out, fin, kept = kda.glr_fwd(x, x, ls, keep=True)
    cut = T - 104  # where a state is kept
    state = kept.view(-1, H, K)[cut // 8].unsqueeze(0)
    tail = x[:, cut:].contiguous()
    want, want_fin = kda.glr_fwd(tail, tail, ls, initial_state=state)
    close(out[:, cut:], want, 512)
    close(fin, want_fin, 512)
    grads = kda.glr_bwd(x, x, out, ls, kept=kept)
    refs = kda.glr_bwd(tail, tail, out[:, cut:].contiguous(), ls, initial_state=state)
    for k in (0, 1):
        close(grads[k][:, cut:], refs[k], 6 * 1024)


def test_norm_past_32_bit_offsets():
    T, D = 300_000, 8192
    y = _far(T, D, BF, 63)
    h, n = kda.block_norm_fwd(y, gate=y, residual=y)
    want = kda.block_norm_fwd(y[:, -50:].contiguous(), gate=y[:, -50:].contiguous(), residual=y[:, -50:].contiguous())
    assert torch.equal(h[:, -50:], want[0]) and torch.equal(n[:, -50:], want[1])
    got = kda.block_norm_bwd(y, y, d_n=n, h=h, gate=y)
    ref_ = kda.block_norm_bwd(y[:, -50:].contiguous(), y[:, -50:].contiguous(), d_n=want[1], h=want[0], gate=y[:, -50:].contiguous())
    for k in range(3):
        assert torch.equal(got[k][:, -50:], ref_[k])


# --------------------------------------------------------------------------- nothing to do

@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("cu", [None, [0], [0, 0, 0]])
def test_no_rows(dtype, cu):
    """Batches without a row: states are handed on, their gradients handed back, sums are zeros."""
    B, N = (1, len(cu) - 1) if cu else (2, 2)
    off = torch.tensor(cu, dtype=torch.int32, device="cuda") if cu else None
    r = gen(70)
    x, w, b, s = torch.zeros(B, 0, 20, dtype=dtype, device="cuda"), gpu(r(20, 3)), gpu(r(20)), gpu(r(N, 2, 20).to(dtype))
    out, fin = kda.short_conv_fwd(x, w, b, s, cu_seqlens=off)
    assert out.shape == x.shape and torch.equal(fin, s) and not kda.short_conv_fwd(x, w, b, cu_seqlens=off)[1].any()
    dx, dw, db, ds = kda.short_conv_bwd(x, w, x, b, s, d_final_state=s, cu_seqlens=off)
    assert dx.shape == x.shape and not dw.any() and not db.any() and torch.equal(ds, s)
    X, ls, bi, s0 = x.unflatten(2, (2, 10)), gpu(r(2)), gpu(r(2, 10)), gpu(r(N, 2, 10))
    out, fin, kept = kda.glr_fwd(X, X, ls, bi, X, initial_state=s0, cu_seqlens=off, keep=True)
    assert out.shape == X.shape and torch.equal(fin, s0) and not kept.numel()
    dx, dg, di, da, db, ds = kda.glr_bwd(X, X, X, ls, bi, X, initial_state=s0, d_final_state=s0, cu_seqlens=off, kept=kept)
    assert not da.any() and not db.any() and torch.equal(ds, s0) and di.shape == X.shape
    y, wa = torch.zeros(0, 3, 16, dtype=dtype, device="cuda"), torch.ones(16, device="cuda")
    h, n = kda.block_norm_fwd(y, y, y, wa, wa)
    assert h.shape == y.shape and n.shape == y.shape
    got = kda.block_norm_bwd(y, y, y, y, y, wa, wa)
    assert not got[3].any() and not got[4].any()
    assert kda.short_conv_step(x, w, s).shape == x.shape if B <= N else True


def test_offsets_out_of_order():
    """Offsets that are out of range or order move boundaries, but every call returns, and what is in order still holds."""
    lens = [50, 30, 20]
    x, w, b, s = map(gpu, conv_case(lens, True, 16, 4, F32, True, True, 71))
    X, z, ls, bi, i, s0 = map(gpu, scan_case(lens, True, 2, 8, F32, True, True, True, 72))
    for bad in ([0, 50, 80, 130], [0, 50, 80, -5], [0, 70, 40, 100], [5, 50, 80, 100], [-9, 50, 1 << 30, 100], [100, 80, 50, 0]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        out, _ = kda.short_conv_fwd(x, w, b, s, cu_seqlens=cu)
        kda.short_conv_bwd(x, w, x, b, s, d_final_state=s, cu_seqlens=cu)
        o, _, kept = kda.glr_fwd(X, z, ls, bi, i, initial_state=s0, cu_seqlens=cu, keep=True)
        kda.glr_bwd(X, z, X, ls, bi, i, initial_state=s0, d_final_state=s0, cu_seqlens=cu, kept=kept)
        torch.cuda.synchronize()
        if bad[:2] == [0, 50] and bad[3] >= 50:
            good = gpu(offsets(lens))
            assert torch.equal(out[:, :50], kda.short_conv_fwd(x, w, b, s, cu_seqlens=good)[0][:, :50])
            assert torch.equal(o[:, :50], kda.glr_fwd(X, z, ls, bi, i, initial_state=s0, cu_seqlens=good)[0][:, :50])


@pytest.mark.parametrize("shape", [(0, 16), (1, 0, 16), (2, 0, 3, 16), (2, 5, 0, 16)])
def test_norm_of_no_rows(shape):
    """A batch without tokens, in every form that has a place for them, recorded and not: empty results, and gradients of the weights that are zeros."""
    y, r, z = (torch.empty(shape, dtype=BF, device="cuda", requires_grad=True) for _ in range(3))
    wa, wb = (torch.ones(16, device="cuda", requires_grad=True) for _ in range(2))
    h, n = kda.block_norm(y, gate=z, residual=r, weight_after=wa, weight_before=wb)
    assert h.shape == shape and n.shape == shape
    dy, dz, dr, da, db = torch.autograd.grad([h, n], [y, z, r, wa, wb], [torch.empty_like(h), torch.empty_like(n)])
    assert dy.shape == shape and dz.shape == shape and dr.shape == shape
    assert torch.equal(da, torch.zeros_like(wa)) and torch.equal(db, torch.zeros_like(wb))
    assert kda.gated_norm(y.detach(), z.detach(), wa.detach()).shape == shape


def test_refusals_name_what_to_call():
    x = torch.zeros(2, 3, 1, 8, device="cuda")
    for call in (lambda: kda.glr_step([1.0], x, x[0]), lambda: kda.glr_step(x, None, x[0]), lambda: kda.glr_step(x, x, x[0], in_gate=1.0)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError, match="short_conv"):
        kda.short_conv_fwd(x[:, :, 0].requires_grad_(), torch.zeros(8, 2, device="cuda"))


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("T", [40, 400, 3000])
def test_scan_does_not_forget_what_is_not_finite(bad, T):
    """alpha = e^-5 everywhere: a tile's product of decays leaves float32's range, but inf * alpha stays inf and NaN stays
    NaN down the sequence (through zero decays at most inf * 0, NaN), as in the recurrence row by row; the next sequence and the other
    channels have none of it.  Its gradients: the same from the right."""
    H, K, behind = 2, 8, 30
    gate = torch.full((1, T + behind, H, K), -5.0, device="cuda")
    x = torch.ones(1, T + behind, H, K, device="cuda")
    s0 = torch.zeros(2, H, K, device="cuda")
    s0[0, 1, 3] = bad
    cu = gpu(torch.tensor([0, T, T + behind], dtype=torch.int32))
    out, final, kept = kda.glr_fwd(x, gate, initial_state=s0, cu_seqlens=cu, keep=True)
    want = torch.ones_like(out, dtype=torch.bool)
    want[:, :T, 1, 3] = False
    assert torch.equal(torch.isfinite(out), want)
    assert not torch.isfinite(final[0, 1, 3]) and torch.isfinite(final).sum() == final.numel() - 1
    d_final = torch.zeros_like(final)
    d_final[0, 1, 3] = bad
    dx, dg, _, _, _, ds = kda.glr_bwd(x, gate, torch.ones_like(x), initial_state=torch.zeros_like(s0), d_final_state=d_final, cu_seqlens=cu)
    assert torch.equal(torch.isfinite(dx), want) and torch.equal(torch.isfinite(dg), want)
    assert not torch.isfinite(ds[0, 1, 3]) and torch.isfinite(ds).sum() == ds.numel() - 1


@pytest.mark.parametrize("lens,H,K", [([20] * 6, 2, 4), ([20] * 10, 2, 4), ([12] * 20, 3, 5), ([37] * 70, 1, 8), ([37] * 30, 4, 258)])
@pytest.mark.parametrize("logits", [True, False])
def test_no_sequence_reaches_another_over_tiles(lens, H, K, logits):
    """What is not finite in one input of one sequence changes no bit of any other, forward or backward: several
    beginnings in tiles of their own on both sides of it, 15 tiles (joined by their readers) and more (joined by a pass over
    them, some with several tiles to a group of lanes, some with more than 1024 channels)."""
    N, T = len(lens), sum(lens)
    x, z, ls, b, i, s = scan_case(lens, True, H, K, F32, logits, True, True, 80)
    r = gen(81)
    data = dict(x=x, gate=z, in_gate=i, initial_state=s, d_out=r(*x.shape), d_final_state=r(N, H, K))
    cu, ls, b = gpu(offsets(lens)), gpu(ls), gpu(b)

    def run(x, gate, in_gate, initial_state, d_out, d_final_state):
        kw = dict(log_scale=ls, bias=b, in_gate=in_gate, initial_state=initial_state, cu_seqlens=cu)
        out, final, kept = kda.glr_fwd(x, gate, keep=True, **kw)
        dx, dg, di, _, _, ds = kda.glr_bwd(x, gate, d_out, d_final_state=d_final_state, kept=kept, **kw)
        return [out, dx, dg, di], [final, ds]

    data = {k: gpu(v) for k, v in data.items()}
    rows, states = run(**data)
    for n in (0, N // 3, N // 2, N - 1):
        at = offsets(lens)[n].item()
        mine = torch.zeros(T, dtype=torch.bool, device="cuda")
        mine[at : at + lens[n]] = True
        others = torch.arange(N, device="cuda") != n
        for what, bad in [(k, v) for k in data for v in (float("nan"), float("inf")) if k != "gate" or v != v]:
            new = {k: v.clone() for k, v in data.items()}
            if what in ("initial_state", "d_final_state"):
                new[what][n] = bad
            else:
                new[what][0, at + 5] = bad
            got_rows, got_states = run(**new)
            for k, (u, v) in enumerate(zip(got_rows, rows)):
                assert torch.equal(u[:, ~mine], v[:, ~mine]), (n, what, bad, k)
            for k, (u, v) in enumerate(zip(got_states, states)):
                assert torch.equal(u[others], v[others]), (n, what, bad, k)
            # the sigmoid of an infinite input gate is 1
            back = what in ("d_out", "d_final_state")
            if (what, bad) != ("in_gate", float("inf")):
                assert not torch.isfinite((got_rows[1] if back else got_rows[0])[:, mine]).all(), (n, what, bad)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("infinite", [False, True])
def test_scan_masked_logits(dtype, sign, infinite):
    """Logits at the end of their type's range, or infinite: the sigmoid is 0 or 1, what they add to a gradient 0 (the limit of u du
    for infinite ones; the 64-bit form has it at the type's largest number).  d log_scale is a sum of 45 x 12 terms, of which those
    of these logits are 0; tolerances as in test_scan, whose decays these are but for alpha = 1."""
    lens, H, K = [30, 0, 15], 2, 12
    x, z, ls, b, i, s = scan_case(lens, True, H, K, dtype, True, True, True, 82)
    far = sign * torch.finfo(dtype).max
    for at in (0, 7, 29, 30, 44):
        z[0, at, at % 2, 3 : 3 + at % 5] = far
    zs = z.clone()
    if infinite:
        zs[z == far] = sign * float("inf")
    d_out, d_fin = gen(83)(*x.shape).to(dtype), gen(84)(3, H, K)
    cu = gpu(offsets(lens))
    kw = dict(log_scale=gpu(ls), bias=gpu(b), in_gate=gpu(i), initial_state=gpu(s), cu_seqlens=cu)
    out, fin = kda.glr_fwd(gpu(x), gpu(zs), **kw)
    want, want_fin = ref.scan(f64(x), f64(z), f64(ls), f64(b), f64(i), f64(s), lens, True)
    close(out, want, 512, "out")
    close(fin, want_fin, 512, "final")
    got = kda.glr_bwd(gpu(x), gpu(zs), gpu(d_out), d_final_state=gpu(d_fin), **kw)
    assert all(torch.isfinite(g).all() for g in got)
    assert not got[1][gpu(z) == far].any()
    # the formula's gradient, its own rows with alpha = 1 left out (the root has no derivative there, which counts as 0)
    g = ref.decay(f64(z), f64(ls), f64(b))
    a, f, gi = torch.exp(g), torch.sqrt(-torch.expm1(2 * g)), torch.sigmoid(f64(i))
    lam, before = torch.zeros(45, H, K).double(), torch.zeros(45, H, K).double()
    for first, last, n in ((0, 30, 0), (30, 45, 2)):
        h, m = f64(s)[n], f64(d_fin)[n]
        for t in range(first, last):
            before[t] = h
            h = a[0, t] * h + (f * gi * f64(x))[0, t]
        for t in reversed(range(first, last)):
            lam[t] = f64(d_out)[0, t] + m
            m = a[0, t] * lam[t]
    dg = lam * (a[0] * before - torch.where(f > 0, gi * f64(x) * a * a / f.clamp_min(1e-300), 0 * f)[0])
    u = torch.exp(f64(ls))[:, None] * (f64(z) + f64(b))
    du = dg * (-5 * torch.sigmoid(u) * torch.sigmoid(-u))[0]
    terms = (du * u[0].clamp(-40, 40)).pow(2).sum().sqrt()
    assert float((f64(got[3]) - (du * u[0]).sum((0, 2))).abs().max()) <= (6 * 1024 + 4 * (45 * K) ** 0.5) * 2.0 ** -24 * max(1.0, float(terms))
    close(got[4], (du * torch.exp(f64(ls))[:, None]).sum(0), 6 * 1024 + 4 * 45 ** 0.5, "d bias", 1.0)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [8, 33, 264, 4104, 16384])
@pytest.mark.parametrize("gate", [False, True])
def test_norm_gradient_without_norm_after_is_not_of_y(dtype, D, gate):
    """h = scale sigmoid(gate) y: the gradient of y is scale sigmoid(gate) d_h, whatever y holds; each product and the sigmoid's three
    operations round once, and the result to its type."""
    r = gen(85)
    y, z, d = r(6, D).to(dtype), r(6, D).to(dtype) if gate else None, r(6, D).to(dtype)
    y[1, D // 2], y[3, 0], y[4, D - 1] = float("inf"), -float("inf"), float("nan")
    dy, dz, dr, _, _ = kda.block_norm_bwd(gpu(y), gpu(d), gate=gpu(z), norm_after=False, norm_before=False, scale=0.5)
    close(dy, 0.5 * f64(d) * (torch.sigmoid(f64(z)) if gate else 1), 16, "dy")
    assert torch.equal(dr, gpu(d))
    if gate:  # of y itself, its own number alone
        assert torch.equal(torch.isfinite(dz), torch.isfinite(gpu(y)))


def test_forward_mode_is_refused_by_every_input():
    """Weights, gates, states and buffers with a tangent, and recorded calls with one beside a leaf that requires grad."""
    from torch.autograd import forward_ad
    dual = lambda t: forward_ad.make_dual(t, torch.ones_like(t))  # noqa: E731
    x, X, w, ls, s = (torch.zeros(*n, device="cuda") for n in ((1, 4, 32), (1, 4, 2, 16), (32, 4), (2,), (1, 2, 16)))
    leaf, Leaf = x.clone().requires_grad_(), X.clone().requires_grad_()
    with forward_ad.dual_level():
        for call in (lambda: kda.short_conv(x, dual(w)), lambda: kda.short_conv_step(x, w, dual(torch.zeros(1, 3, 32, device="cuda"))), lambda: kda.glr_fwd(X, dual(X)),
                     lambda: kda.glr_fwd(X, X, ls, initial_state=dual(s)), lambda: kda.glr_fwd(X, X, in_gate=dual(X)[..., :8]), lambda: kda.glr_step(X, X, dual(s)),
                     lambda: kda.block_norm(X, gate=dual(X)), lambda: kda.block_norm(X, residual=dual(X)), lambda: kda.block_norm(X, weight_before=dual(X[0, 0, 0])),
                     lambda: kda.glr_fwd(X, X, out=dual(X.clone()))):
            with pytest.raises(ValueError, match="forward-mode tangent"):
                call()
        for call in (lambda: kda.short_conv(leaf, dual(w)), lambda: kda.gated_linear_recurrence(Leaf, dual(X)), lambda: kda.block_norm(Leaf, residual=dual(X)),
                     lambda: kda.gated_norm(dual(Leaf))):
            with pytest.raises(NotImplementedError):
                call()
        assert not kda.short_conv(leaf, w)[0].any() and not kda.block_norm(X)[0].any()  # what has none goes on as before


@pytest.mark.parametrize("many", [70, 5000])
def test_batch_padded_with_empty_sequences(many):
    """Thousands of sequences without rows, in front, in the middle and at the end, change nothing of the others, and hand their states on."""
    lens = [37, 100, 1, 62]
    x, w, b, s = map(gpu, conv_case(lens, True, 20, 4, BF, True, True, 86))
    X, z, ls, bi, i, s0 = map(gpu, scan_case(lens, True, 2, 10, F32, True, True, True, 87))
    padded = [0] * many + lens[:2] + [0] * many + lens[2:] + [0] * many
    real = torch.tensor([k for k, n in enumerate(padded) if n], device="cuda")
    cu, few = gpu(offsets(padded)), gpu(offsets(lens))

    def spread(t):
        more = gpu(gen(88)(len(padded), *t.shape[1:]).to(t.dtype))
        more[real] = t
        return more
    s_, s0_ = spread(s), spread(s0)
    empty = torch.tensor([n == 0 for n in padded], device="cuda")
    for got, want, handed in (
            (kda.short_conv_fwd(x, w, b, s_, cu_seqlens=cu), kda.short_conv_fwd(x, w, b, s, cu_seqlens=few), s_),
            (kda.glr_fwd(X, z, ls, bi, i, initial_state=s0_, cu_seqlens=cu), kda.glr_fwd(X, z, ls, bi, i, initial_state=s0, cu_seqlens=few), s0_)):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1][real], want[1]) and torch.equal(got[1][empty], handed[empty])
    for got, want, handed in (
            (kda.short_conv_bwd(x, w, x, b, s_, d_final_state=s_, cu_seqlens=cu), kda.short_conv_bwd(x, w, x, b, s, d_final_state=s, cu_seqlens=few), s_),
            (kda.glr_bwd(X, z, X, ls, bi, i, initial_state=s0_, d_final_state=s0_, cu_seqlens=cu), kda.glr_bwd(X, z, X, ls, bi, i, initial_state=s0, d_final_state=s0, cu_seqlens=few), s0_)):
        for u, v in zip(got[:-1], want[:-1]):
            assert torch.equal(u, v)
        assert torch.equal(got[-1][real], want[-1]) and torch.equal(got[-1][empty], handed[empty])


@pytest.mark.parametrize("dtype", [F32, BF])
def test_recorded_block_in_a_graph(dtype):
    """Forward and backward of the recorded calls, one after another as in a block, captured and replayed with new inputs in place
    between eager passes: every replay gives the eager results' bits.  Thirty rows behind the last sequence."""
    lens, H, K = [60, 70, 0, 30], 2, 24
    T, C, cu = sum(lens) + 30, H * K, gpu(offsets(lens))

    def make(seed):
        r = gen(seed)
        rows = [r(1, T, n).to(dtype) for n in (C, C, 4 * C)]
        return [gpu(t) for t in rows + [r(C, 4) / 2, r(C), 0.2 * r(H), r(H, K), 1 + 0.2 * r(C), 1 + 0.2 * r(K), r(4, 3, C).to(dtype), r(4, H, K)] +
                [r(1, T, C).to(dtype), r(1, T, C).to(dtype), r(4, 3, C).to(dtype), r(4, H, K)]]

    def turn(data):
        leaves = [t.detach().requires_grad_() for t in data[:11]]
        y, x, u, w, b, ls, bias, norm, head, s, s0 = leaves
        h, n = kda.block_norm(y, residual=x, weight_after=norm, weight_before=norm, scale=0.5, silu=True)
        v, rows = kda.short_conv(u[..., :C] + n, w, b, s, cu_seqlens=cu)
        part = lambda k: u[..., k * C : (k + 1) * C].unflatten(-1, (H, K))  # noqa: E731
        o, state = kda.gated_linear_recurrence(v.unflatten(-1, (H, K)), part(1), ls, bias, part(2), initial_state=s0, cu_seqlens=cu)
        outs = [h, kda.gated_norm(o, part(3), head).flatten(-2), rows, state]
        return outs + list(torch.autograd.grad(outs, leaves, data[11:]))
    static = make(90)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        turn(static)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = turn(static)
    for seed in (91, 92, 93):
        new = make(seed)
        for t, m in zip(static, new):
            t.copy_(m)
        graph.replay()
        torch.cuda.synchronize()
        want = turn(new)
        torch.cuda.synchronize()
        for k, (p, q) in enumerate(zip(got, want)):
            assert torch.isfinite(p).all() and torch.equal(p, q), k
