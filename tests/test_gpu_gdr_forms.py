"""GPU parity of the gated delta rule in the forms and at the sizes that it is trained and served
with: the bits that a float32 output keeps, two column tiles a workgroup at full width, mixed
types, packed batches that are padded behind their last sequence.

Tolerances, from the roundings that the kernels make.  Operands of the matrix cores are exact
(bf16 inputs) or off by at most 2^-24 of the value (three bf16 parts), accumulators and the rest
are float32, whose roundings are at most 2^-24 and, as they are independent, 2^-24 / sqrt(3) = 3.4e-8
in the mean square.  On the way to a chunk's end state stand about 40 of them (12 matrix instructions
and a scaling for X, 12 for M (beta X), 6 for K^T E, the cuts and the decays), as many in M itself,
and 30 more on the way to an output (12 for Q S, 12 for P Vn, the cuts, three factors): sqrt(110)
3.4e-8 = 3.6e-7 of the partial sums, which are somewhat larger than what they end as.  NORM, 1e-6 of
an output's or a state's 2-norm, leaves a factor of three for that.  An operand of two parts (16 bits) is
off by 2^-16 at most and 2^-18 = 3.8e-6 in the mean square, and does not pass it.  The largest element
is held to 1e-5, as with float32 inputs elsewhere.
"""
import numpy as np
import pytest
import torch

import gated_delta_rule_31_amd as kda
from tests import gdr_reference as ref
from tests.helpers import err_fp32, f64
from tests.test_gpu_gdr import NAMES, _bwd_check, _cotangents, _fwd, _gpu, _norm

pytestmark = pytest.mark.gpu

NORM = 1e-6


def _full_bits(out, final, want, what=""):
    for name, x, y in (("out", out, want[0]), ("state", final, want[1])):
        assert x.dtype == torch.float32 and np.all(np.isfinite(f64(x))), (what, name)
        n, e = _norm(x, y), err_fp32(x, y)
        assert n <= NORM and e <= 1e-5, "%s %s: %.2e in norm, %.2e" % (what, name, n, e)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("HK,HV,K,V,lens", [(2, 4, 128, 128, None), (1, 3, 16, 16, None), (1, 2, 32, 64, None), (2, 2, 64, 32, [70, 0, 129, 1])])
def test_fwd_float32_output_keeps_24_bits(dtype, HK, HV, K, V, lens):
    """The state's part of an output, the chunk's own and both, with inputs in either type."""
    i = ref.make(1, 200, HK, HV, K, V, dtype, seed=50 + K, seqlens=lens)
    out, final = _fwd(i, K ** -0.5, out_dtype=torch.float32)
    _full_bits(out, final, ref.scan(i, K ** -0.5))


# ------------------------------------------------------------------- packed and padded to a bucket

def _padded(T, used, HK, HV, K, V, dtype, seed, cuts=(0.3, 0.55)):
    """A packed batch of three sequences in the first `used` rows of T: what lies behind them is what was there before."""
    lens = np.diff([0] + [int(used * c) for c in cuts] + [used])
    i = ref.make(1, used, HK, HV, K, V, dtype, seed=seed, seqlens=list(lens))
    d = _gpu(i)
    more = lambda x: torch.cat([x, x.new_full((1, T - used, *x.shape[2:]), float("nan"))], 1)  # noqa: E731
    d_out, d_fin = _cotangents(i, seed + 1, dtype)
    return d, {n: more(d[n]) for n in ("q", "k", "v", "g", "beta")}, d_out.cuda(), more(d_out.cuda()), d_fin.cuda()


@pytest.mark.parametrize("T,used", [(129, 0), (64, 1), (65, 1), (200, 199), (192, 130), (192, 128), (640, 65), (1000, 63)])
@pytest.mark.parametrize("dtype,grad,HK,HV,K,V", [(torch.bfloat16, torch.bfloat16, 2, 4, 128, 128), (torch.float32, torch.float32, 1, 3, 16, 16),
                                                  (torch.bfloat16, torch.float32, 1, 70, 32, 64)])
def test_bwd_padded_bucket(T, used, dtype, grad, HK, HV, K, V):
    """Gradients behind the last sequence are zeros, and those of its rows the ones of the batch without them, at
    tails that end inside a chunk, begin inside one, and are all there is."""
    d, wide, d_out, wide_out, d_fin = _padded(T, used, HK, HV, K, V, dtype, T + used)
    kw = dict(initial_state=d["s0"], d_final_state=d_fin, cu_seqlens=d["cu"], grad_dtype=grad)
    got = kda.gdr_chunk_bwd(*wide.values(), wide_out, **kw)
    want = kda.gdr_chunk_bwd(*[d[n] for n in wide], d_out, **kw)
    for name, x, y in zip(NAMES[:5], got, want):
        assert torch.equal(x[:, :used], y), name
        assert not x[:, used:].any(), name  # NaN counts as something
    assert torch.equal(got[5], want[5] if used else d_fin)


def test_bwd_padding_is_not_the_call():
    """A bucket of which an eighth is used costs less than a full one (the slots without a chunk clear the rest)."""
    def call(used):
        _, wide, _, d_out, d_fin = (x for x in _padded(8192, used, 16, 32, 128, 128, torch.bfloat16, 60))
        cu = torch.tensor([0, used // 3, used], dtype=torch.int32, device="cuda")
        wide = {n: x.nan_to_num() for n, x in wide.items()}
        return lambda: kda.gdr_chunk_bwd(*wide.values(), d_out.nan_to_num(), cu_seqlens=cu)

    def time(f):
        out = []
        for _ in range(7):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            f()
            b.record()
            b.synchronize()
            out.append(a.elapsed_time(b))
        return sorted(out)[3]
    few, full = time(call(1000)), time(call(8191))
    print("1000 of 8192 rows %.0f us, 8191 %.0f us" % (1e3 * few, 1e3 * full))
    assert few < full


def test_gated_delta_rule_is_one_function_recorded_or_not():
    """A padded packed batch gives the same rows, those behind the last sequence among them, in training, without
    gradients and under no_grad, whatever the memory held that the output is made in."""
    d, wide, _, _, _ = _padded(300, 130, 2, 4, 32, 64, torch.bfloat16, 70)
    leaves = [x.clone().requires_grad_() for x in wide.values()]

    def fresh(f):
        gone = [torch.full_like(wide["v"], float("nan")) for _ in range(4)]  # what the next outputs are made in
        del gone
        return f()
    call = lambda xs: kda.gated_delta_rule(*xs, initial_state=d["s0"], cu_seqlens=d["cu"], scale=0.5)  # noqa: E731
    recorded = fresh(lambda: call(leaves))
    assert recorded[0].requires_grad
    with torch.no_grad():
        under = fresh(lambda: call(leaves))
    plain = fresh(lambda: call(list(wide.values())))
    for out, fin in (under, plain):
        assert not out.requires_grad and torch.equal(out, recorded[0]) and torch.equal(fin, recorded[1])
    assert not plain[0][:, 130:].any() and plain[0][:, :130].any()


# ------------------------------------------------------------------- views off a 16-byte border

def _off(x, n=1):
    """x's values n elements behind a 16-byte border."""
    flat = torch.empty(x.numel() + n, dtype=x.dtype, device="cuda")
    flat[n:] = x.reshape(-1)
    return flat[n:].reshape(x.shape)


@pytest.mark.parametrize("drawn", [True, False])
def test_verify_takes_views_as_they_are(drawn):
    """Requests behind the first of an odd vocabulary start off a 16-byte border: nothing of them is copied."""
    gen = torch.Generator(device="cuda").manual_seed(80)
    B, D, vocab = 6, 2, 50001
    p = torch.softmax(2 * torch.randn(B + 1, D + 1, vocab, generator=gen, device="cuda"), -1)[1:]
    q = torch.softmax(2 * torch.randn(B + 1, D, vocab, generator=gen, device="cuda"), -1)[1:]
    x = torch.randint(0, vocab, (B + 1, D), generator=gen, device="cuda").to(torch.int32)[1:]
    u = torch.rand(B + 1, D + 1, generator=gen, device="cuda")[1:]
    n = torch.tensor([9, 2, 2, 1, 0, 3, 2], dtype=torch.int32, device="cuda")[1:]
    assert p.data_ptr() % 16 and n.data_ptr() % 16
    kw = dict(draft_probs=q if drawn else None, lengths=n)
    kda.draft_verify(p, x, u, **kw)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    tokens, accepted = kda.draft_verify(p, x, u, **kw)
    assert torch.cuda.max_memory_allocated() - before < 1 << 20
    wt, wa = ref.verify(p.cpu(), x.cpu(), u.cpu(), q.cpu() if drawn else None, n.cpu())
    assert np.array_equal(tokens.cpu().numpy(), wt) and np.array_equal(accepted.cpu().numpy(), wa)


def test_calls_take_numbers_off_the_border():
    """What is read number by number (decays and strengths per head, offsets, slots, lengths) may start on any
    element; decays per channel, which are read in wide loads, are moved to a border."""
    d = _gpu(ref.make(1, 130, 2, 4, 32, 32, torch.bfloat16, seed=81, seqlens=[70, 60]))
    d_out, d_fin = _cotangents(d, 82)
    args = [d[n] for n in ("q", "k", "v", "g", "beta")]
    off = args[:3] + [_off(d["g"]), _off(d["beta"], 3)]
    for f, more in ((kda.gdr_chunk_fwd, ()), (kda.gdr_chunk_bwd, (d_out.cuda(),))):
        want = f(*args, *more, initial_state=d["s0"], cu_seqlens=d["cu"])
        got = f(*off, *more, initial_state=d["s0"], cu_seqlens=_off(d["cu"]))
        assert all(torch.equal(x, y) for x, y in zip(want, got))
    for channels in (False, True):
        q, k, v, beta = (d[n][0, :9].reshape(3, 3, *d[n].shape[2:]).contiguous() for n in ("q", "k", "v", "beta"))
        g = -torch.rand(3, 3, 4, *((32,) if channels else ()), device="cuda")
        slots = torch.arange(9, dtype=torch.int32, device="cuda").reshape(3, 3)
        start, lengths = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 2, 1], [3, 1, 2]))
        states = torch.randn(9, 4, 32, 32, device="cuda")
        a, b = states.clone(), states.clone()
        want = kda.gdr_recurrent_step(q, k, v, g, beta, a, slots=slots, start=start, lengths=lengths)
        got = kda.gdr_recurrent_step(q, k, v, _off(g), _off(beta), b, slots=_off(slots), start=_off(start, 3), lengths=_off(lengths, 2))
        assert torch.equal(want, got) and torch.equal(a, b)


def test_verify_uniforms_outside_their_range():
    """1 or more draws the last token that has weight; NaN or less than 0 the first, and no draft holds against NaN."""
    nan, inf = float("nan"), float("inf")
    p = torch.tensor([0, 0.25, 0.5, 0.25, 0]).expand(8, 2, 5).contiguous().cuda()
    x = torch.full((8, 1), 2, dtype=torch.int32, device="cuda")
    #                   draft 2 holds while u < p(2) = 0.5; refused, the residual is p without token 2
    u = torch.tensor([[0.0, nan], [0.0, -1.0], [0.0, 1.0], [0.0, inf], [0.0, -inf], [nan, 0.0], [nan, nan], [nan, 7.0]], device="cuda")
    tokens, accepted = kda.draft_verify(p, x, u)
    assert accepted.tolist() == [1, 1, 1, 1, 1, 0, 0, 0]
    assert tokens.tolist() == [[2, 1], [2, 1], [2, 3], [2, 3], [2, 1], [1, -1], [1, -1], [3, -1]]


# ------------------------------------------------------------------- full widths, mixed types, long calls

def _rounded_once(got, want, rest, what=""):
    """An output in bfloat16: half a step of the value, 2^-8, beside what the float32 one is held to."""
    rms = np.sqrt(np.mean(want ** 2))
    assert got.dtype == torch.bfloat16 and np.all(np.isfinite(f64(got))), what
    over = np.abs(f64(got) - want) - 2.0 ** -8 * np.abs(want) - rest * np.maximum(np.abs(want), rms)
    assert over.max() <= 0, "%s: %.2e over" % (what, over.max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("HK,HV,K,V,lens", [(24, 72, 128, 128, None), (16, 32, 128, 128, [70, 60]), (9, 36, 64, 128, [64, 1, 0, 65]), (33, 132, 16, 64, None)])
def test_fwd_two_column_tiles(dtype, HK, HV, K, V, lens):
    """Sequences x heads x 16-column tiles of at least twice the compute units (256): two tiles a workgroup."""
    i = ref.make(1, 130, HK, HV, K, V, dtype, seed=90 + K, seqlens=lens)
    assert i["N"] * HV * (V // 16) >= 512
    out, final = _fwd(i, K ** -0.5, out_dtype=torch.float32)
    want = ref.scan(i, K ** -0.5)
    _full_bits(out, final, want)
    out, _ = _fwd(i, K ** -0.5, out_dtype=torch.bfloat16)
    _rounded_once(out, want[0], 1e-5, "bf16 out")


@pytest.mark.parametrize("K,V", [(16, 128), (32, 16), (64, 64), (128, 128)])
def test_fwd_float32_inputs_bfloat16_output(K, V):
    i = ref.make(2, 100, 2, 4, K, V, torch.float32, seed=100 + K)
    out, final = _fwd(i, 0.5, out_dtype=torch.bfloat16)
    want = ref.scan(i, 0.5)
    _rounded_once(out, want[0], 1e-5)
    assert err_fp32(final, want[1]) <= 1e-5


@pytest.mark.parametrize("dtype,HK,HV", [(torch.bfloat16, 24, 72), (torch.float32, 8, 24), (torch.float32, 1, 2)])
def test_fwd_long(dtype, HK, HV):
    """Twenty-four chunks, the last one cut: the first and the last key head's value heads against the definition."""
    i = ref.make(1, 1500, HK, HV, 128, 128, dtype, seed=110 + HV, decay=(0.002, 1.0))
    out, final = _fwd(i, 128 ** -0.5, out_dtype=torch.float32)
    for h in {0, HK - 1}:
        some = slice(h * HV // HK, (h + 1) * HV // HK)
        part = {**i, "q": i["q"][:, :, h : h + 1], "k": i["k"][:, :, h : h + 1], "s0": i["s0"][:, some], **{n: i[n][:, :, some] for n in ("v", "g", "beta")}}
        _full_bits(out[:, :, some], final[:, some], ref.scan(part, 128 ** -0.5), "key head %d" % h)


@pytest.mark.parametrize("HK,HV,K,V", [(2, 4, 16, 32), (1, 3, 32, 16), (2, 2, 64, 64), (2, 4, 128, 128), (33, 132, 64, 64), (33, 132, 128, 64)])
def test_bwd_float32_inputs_bfloat16_cotangents(HK, HV, K, V):
    _bwd_check(ref.make(1, 70, HK, HV, K, V, torch.float32, seed=120 + K), 121, 0.5, torch.bfloat16)


@pytest.mark.parametrize("K,V,HK,HV", [(128, 128, 2, 4), (64, 128, 1, 3), (16, 16, 2, 2), (128, 128, 16, 32)])
def test_bwd_packed_bfloat16(K, V, HK, HV):
    lens = [70, 0, 1, 64, 130] if HV < 32 else [66, 64]
    _bwd_check(ref.make(1, sum(lens), HK, HV, K, V, torch.bfloat16, seed=130 + K + HV, seqlens=lens), 131, K ** -0.5, torch.bfloat16)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("K,V,lens", [(128, 128, None), (32, 64, [70, 0, 61]), (16, 16, None)])
def test_bwd_bfloat16_gradients(dtype, K, V, lens):
    """Gradients written in bfloat16 (dq, dk, dv; dg, dbeta and the state's stay float32) against the definition's."""
    i = ref.make(1, 131, 2, 4, K, V, dtype, seed=140 + K, seqlens=lens)
    d_out, d_fin = _cotangents(i, 141, dtype)
    d = _gpu(i)
    got = kda.gdr_chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["beta"], d_out.cuda(), initial_state=d["s0"], d_final_state=d_fin.cuda(),
                            cu_seqlens=d["cu"], scale=0.5, grad_dtype=torch.bfloat16)
    want = ref.scan_bwd(i, d_out, d_fin, 0.5)
    for name, x, y in zip(NAMES, got, want):
        if name in ("dq", "dk", "dv"):
            _rounded_once(x, y, 5e-5, name)
        else:
            assert x.dtype == torch.float32 and err_fp32(x, y) <= 5e-5, name


# ------------------------------------------------------------------- offsets past 32 bits

def test_long_rows_pass_32_bits():
    """More than 2^31 elements of v, and a workspace beyond 2^32 bytes: the last tokens' outputs and gradients are bit
    for bit those of a call that starts from the state before them (on a chunk's border), and the first tokens'
    gradients those of a call that ends there."""
    HK, HV, K, V, tail = 2, 64, 16, 128, 129
    head = (1 << 31) // (HV * V) // 64 * 64 + 64
    T = head + tail
    assert head * HV * V > 1 << 31
    gen = torch.Generator(device="cuda").manual_seed(150)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    unit = lambda x: (x / x.norm(dim=-1, keepdim=True)).to(torch.bfloat16)  # noqa: E731
    v, d_out = (torch.empty(1, T, HV, V, dtype=torch.bfloat16, device="cuda").normal_(generator=gen) for _ in range(2))
    args = [unit(rand(1, T, HK, K)), unit(rand(1, T, HK, K)), v, -0.05 * rand(1, T, HV).abs(), torch.sigmoid(rand(1, T, HV))]
    first, last = [x[:, :head] for x in args], [x[:, head:] for x in args]
    d_fin = rand(1, HV, K, V)
    out, fin = kda.gdr_chunk_fwd(*args)
    _, mid = kda.gdr_chunk_fwd(*first)
    o, f = kda.gdr_chunk_fwd(*last, initial_state=mid)
    assert torch.equal(out[:, head:], o) and torch.equal(fin, f)
    del out, o
    tail_grads = kda.gdr_chunk_bwd(*last, d_out[:, head:], initial_state=mid, d_final_state=d_fin)
    grads = kda.gdr_chunk_bwd(*args, d_out, d_final_state=d_fin)
    assert all(torch.equal(x[:, head:], y) for x, y in zip(grads[:5], tail_grads))
    head_grads = kda.gdr_chunk_bwd(*first, d_out[:, :head], d_final_state=tail_grads[5])
    assert all(torch.equal(x[:, :head], y) for x, y in zip(grads[:5], head_grads)) and torch.equal(grads[5], head_grads[5])
    # and the first tokens are the definition's
    i = dict(zip(("q", "k", "v", "g", "beta"), (x[:, :130].cpu() for x in args)), s0=None, cu=None, N=1)
    now, _ = kda.gdr_chunk_fwd(*args, output_final_state=False)
    _rounded_once(now[:, :130], ref.scan(i)[0], 1e-5)


def test_step_in_a_large_pool():
    """Slots whose states lie beyond 2^31 elements, and 2^33 bytes, into the pool."""
    HV, K, V = 64, 128, 128
    pool = (1 << 31) // (HV * K * V) + 9
    i = ref.make(3, 2, 32, HV, K, V, torch.bfloat16, seed=151, state=False)
    d = _gpu(i)
    states = torch.empty(pool, HV, K, V, device="cuda")
    slots = torch.tensor([[pool - 1, pool - 2], [0, pool - 3], [pool - 4, 1]], dtype=torch.int32)
    where = slots.reshape(-1).long()
    few = 0.3 * torch.randn(6, HV, K, V, generator=torch.Generator().manual_seed(152))
    states[where.cuda()] = few.cuda()
    out = kda.gdr_recurrent_step(d["q"], d["k"], d["v"], d["g"], d["beta"], states, slots=slots.cuda(), out_dtype=torch.float32)
    wo, ws = ref.step(i["q"], i["k"], i["v"], i["g"], i["beta"], few, torch.arange(6).reshape(3, 2), None, None)
    assert err_fp32(out, wo) <= 1e-5 and err_fp32(states[where.cuda()], ws) <= 1e-5


# ------------------------------------------------------------------- several calls at once, captured training

def test_bwd_and_step_on_streams_at_once():
    """Gradients and decode steps that overlap in time on four streams, each with its own workspace or pool."""
    cases = []
    for n in range(4):
        i = ref.make(1, 200 + 70 * n, 2, 4, 64, 64, torch.bfloat16, seed=160 + n, seqlens=[90, 110 + 70 * n])
        d_out, d_fin = _cotangents(i, 161 + n, torch.bfloat16)
        cases.append((_gpu(i), d_out.cuda(), d_fin.cuda()))

    def call(c, states):
        d, d_out, d_fin = c
        args = [d[n] for n in ("q", "k", "v", "g", "beta")]
        grads = kda.gdr_chunk_bwd(*args, d_out, initial_state=d["s0"], d_final_state=d_fin, cu_seqlens=d["cu"])
        return grads + (kda.gdr_recurrent_step(*[x[:, :3] for x in args], states), states)
    want = [call(c, c[0]["s0"][:1].clone()) for c in cases]
    pools = [[c[0]["s0"][:1].clone() for c in cases] for _ in range(5)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in cases], []
    for states in pools:
        for c, s, st in zip(cases, states, streams):
            with torch.cuda.stream(st):
                got.append(call(c, s))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for n, g in enumerate(got) for x, y in zip(g, want[n % 4]))


def test_recorded_call_in_a_graph():
    """A forward and backward pass through autograd, captured, replayed with new inputs in place between eager
    passes: every replay gives the eager gradients."""
    i = _gpu(ref.make(1, 160, 2, 4, 64, 64, torch.bfloat16, seed=170, seqlens=[60, 70, 0, 30]))
    names = ("q", "k", "v", "g", "beta", "s0")
    data = [torch.cat([i[n], i[n][:, :30]], 1) if n != "s0" else i[n] for n in names]  # thirty rows behind the last sequence

    def turn(xs):
        xs = [x.detach().requires_grad_() for x in xs]
        out, fin = kda.gated_delta_rule(*xs[:5], initial_state=xs[5], cu_seqlens=i["cu"], scale=0.5)
        return (out, fin) + torch.autograd.grad([(out.float() ** 2).mean() + fin.square().mean()], xs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        turn(data)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = turn(data)
    for seed in (171, 172, 173):
        new = _gpu(ref.make(1, 160, 2, 4, 64, 64, torch.bfloat16, seed=seed, seqlens=[60, 70, 0, 30]))
        for x, n in zip(data, names):
            (x if n == "s0" else x[:, :160]).copy_(new[n])
        graph.replay()
        torch.cuda.synchronize()
        want = turn(data)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        assert not got[0][:, 160:].any() and all(bool(torch.isfinite(x).all()) for x in got)
