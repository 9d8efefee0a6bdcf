"""CPU checks of the C entry points of what stands around the recurrence in a layer: refusals before any
launch (the pointers are fake), workspace sizes, where sequences begin and end, and the Python
binding's checks; and the 64-bit forms of the GPU tests against differences."""
import os
import subprocess

import pytest
import torch

import gated_delta_rule_31_amd as kda
from gated_delta_rule_31_amd.build import HIPCC
from gated_delta_rule_31_amd.layer import _gate_rows, _rows
from tests import layer_reference as ref


@pytest.fixture(scope="module")
def lib():
    assert os.path.exists(kda.library_path()), "libkda.so is not built"
    return kda._load()


def _conv(lib, x=0x1000, xs=64, dt=1, w=0x2000, b=0x3000, s0=None, sf=None, cu=None, N=0, B=1, T=64, D=64, W=4, fl=8, out=0x4000):
    return lib.kda_short_conv_fwd(x, xs, dt, w, b, s0, sf, cu, N, B, T, D, W, fl, out, None)


BATCH = [(dict(B=-1), 2), (dict(T=-1), 2), (dict(cu=0x900, B=2, N=2), 5), (dict(cu=0x900, N=-1), 5), (dict(cu=0x900, N=0), 5), (dict(T=1 << 31), 4),
         (dict(B=1 << 20, T=1 << 62), 4), (dict(B=1 << 30, T=4), 4)]


@pytest.mark.parametrize("kw,status", BATCH + [
    (dict(D=0), 2), (dict(W=0), 2), (dict(W=1), 4), (dict(W=5), 4), (dict(dt=2), 3), (dict(fl=1), 5), (dict(D=(1 << 20) + 1, xs=1 << 21), 4), (dict(xs=63), 2),
    (dict(x=None), 1), (dict(w=None), 1), (dict(out=None), 1), (dict(out=0x1000), 6), (dict(sf=0x4000), 6), (dict(s0=0x5000, sf=0x5000), 6), (dict(sf=0x3000), 6),
    (dict(x=0x1001), 5), (dict(out=0x4001), 5), (dict(dt=0, x=0x1002), 5), (dict(B=1 << 16, T=1 << 10, D=1 << 20, xs=1 << 20), 4),
    (dict(cu=0x900, N=1 << 30), 4), (dict(T=0, x=None, out=None), 0), (dict(B=0, x=None), 0)])
def test_conv_refusals(lib, kw, status):
    assert _conv(lib, **kw) == status


def _conv_bwd(lib, x=0x1000, xs=64, dt=1, w=0x2000, b=0x3000, s0=None, cu=None, N=0, B=1, T=64, D=64, W=4, fl=8, do=0x4000, dsf=None, dx=0x5000, dw=0x6000,
              db=0x7000, ds0=None, ws=0x8000, wsz=1 << 30):
    return lib.kda_short_conv_bwd(x, xs, dt, w, b, s0, cu, N, B, T, D, W, fl, do, dsf, dx, dw, db, ds0, ws, wsz, None)


@pytest.mark.parametrize("kw,status", BATCH + [
    (dict(W=9), 4), (dict(do=None), 1), (dict(dx=None), 1), (dict(ws=None), 1), (dict(dw=0x1000), 6), (dict(db=0x6000), 6), (dict(ws=0x4000), 6), (dict(ds0=0x900, dsf=0x900), 6),
    (dict(ws=0x8004), 5), (dict(wsz=64), 5), (dict(do=0x4001), 5), (dict(xs=1), 2)])
def test_conv_bwd_refusals(lib, kw, status):
    assert _conv_bwd(lib, **kw) == status


def test_workspaces(lib):
    size = kda.short_conv_bwd_workspace_size
    assert size(torch.bfloat16, 1, 64, 64, 4) == 8 * 5 * 64 * 4  # runs of 8 rows
    assert size(torch.bfloat16, 1, 0, 64, 4) == 0 and size(torch.bfloat16, 1, 64, 64, 5) == 0 and size(torch.bfloat16, 1 << 20, 1 << 62, 64, 4) == 0
    need = size(torch.bfloat16, 1, 64, 64, 4)
    assert _conv_bwd(lib, wsz=need - 1) == 5
    assert kda.glr_kept_size(2, 65, 3, 5) == 17 * 15 * 4  # 130 rows, a state in front of every 8
    assert kda.glr_kept_size(2, 0, 3, 5) == 0 and kda.glr_fwd_workspace_size(0, 5, 1, 1) == 0 and kda.glr_fwd_workspace_size(1, 1 << 31, 1, 1) == 0
    assert kda.glr_bwd_workspace_size(1, 64, 2, 16, True, False) > kda.glr_bwd_workspace_size(1, 64, 2, 16, True, True) > kda.glr_bwd_workspace_size(1, 64, 2, 16, False, True) > 0
    assert _glr(lib, wsz=kda.glr_fwd_workspace_size(1, 64, 2, 16) - 1) == 5
    assert _glr_bwd(lib, wsz=kda.glr_bwd_workspace_size(1, 64, 2, 16, True, True) - 1) == 5
    assert _glr_bwd(lib, kept=None, wsz=kda.glr_bwd_workspace_size(1, 64, 2, 16, True, False) - 1) == 5
    n = kda.block_norm_bwd_workspace_size
    assert n(7, 1, 100) == 7 * 2 * 100 * 4 and n(0, 1, 100) == 0 and n(5, 1, 16385) == 0 and n(1 << 31, 1, 8) == 0
    assert _norm_bwd(lib, wsz=n(64, 2, 16) - 1) == 5


def _glr(lib, x=0x1000, xs=32, dt=1, g=0x2000, gs=32, ls=0x3000, b=0x4000, lb=-5.0, i=0x5000, is_=32, fl=1, s0=None, sf=None, cu=None, N=0, B=1, T=64, H=2, K=16,
         out=0x6000, kept=None, ws=0x7000, wsz=1 << 24):
    return lib.kda_glr_fwd(x, xs, dt, g, gs, ls, b, lb, i, is_, fl, s0, sf, cu, N, B, T, H, K, out, kept, ws, wsz, None)


GATES = [(dict(H=0), 2), (dict(K=0), 2), (dict(dt=3), 3), (dict(fl=2), 5), (dict(lb=0.0), 5), (dict(lb=float("nan")), 5), (dict(ls=None), 5), (dict(H=1 << 15, K=1 << 6), 4)]


@pytest.mark.parametrize("kw,status", BATCH + GATES + [
    (dict(xs=31), 2), (dict(gs=31), 2), (dict(is_=0), 2), (dict(x=None), 1), (dict(g=None), 1), (dict(out=None), 1), (dict(ws=None), 1), (dict(out=0x1000), 6), (dict(kept=0x6000), 6),
    (dict(ws=0x2000), 6), (dict(s0=0x900, sf=0x900), 6), (dict(sf=0x6000), 6), (dict(x=0x1001), 5), (dict(g=0x2001), 5), (dict(ls=None, b=None, g=0x2002), 5), (dict(ws=0x7008), 5),
    (dict(wsz=16), 5), (dict(cu=0x900, N=1 << 30, T=0, x=None, out=None, sf=None), 0), (dict(T=0, x=None, ws=None), 0)])
def test_glr_refusals(lib, kw, status):
    assert _glr(lib, **kw) == status


def _glr_bwd(lib, x=0x1000, xs=32, dt=1, g=0x2000, gs=32, ls=0x3000, b=0x4000, lb=-5.0, i=0x5000, is_=32, fl=1, s0=None, cu=None, N=0, B=1, T=64, H=2, K=16,
             kept=0x6000, do=0x7000, dsf=None, dx=0x8000, dg=0x9000, di=0xa000, dls=0xb000, db=0xc000, ds0=None, ws=0xd000, wsz=1 << 24):
    return lib.kda_glr_bwd(x, xs, dt, g, gs, ls, b, lb, i, is_, fl, s0, cu, N, B, T, H, K, kept, do, dsf, dx, dg, di, dls, db, ds0, ws, wsz, None)


@pytest.mark.parametrize("kw,status", BATCH + GATES + [
    (dict(do=None), 1), (dict(dx=None), 1), (dict(dg=None), 1), (dict(di=None), 1), (dict(ws=None), 1), (dict(dx=0x7000), 6), (dict(ws=0x6000), 6), (dict(db=0xb000), 6),
    (dict(ds0=0x900, dsf=0x900), 6), (dict(ls=None, b=None), 5), (dict(dx=0x8001), 5), (dict(dg=0x9001), 5), (dict(ws=0xd004), 5)])
def test_glr_bwd_refusals(lib, kw, status):
    assert _glr_bwd(lib, **kw) == status


def _norm(lib, y=0x1000, g=0x2000, gs=32, gh=16, dt=1, r=0x3000, ht=1, wa=0x4000, wb=0x5000, n=64, heads=2, D=16, eps=1e-6, fl=3, h=0x6000, o=0x7000):
    return lib.kda_block_norm_fwd(y, g, gs, gh, dt, r, ht, wa, wb, n, heads, D, 1.0, eps, fl, h, o, None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), 2), (dict(heads=0), 2), (dict(D=0), 2), (dict(dt=2), 3), (dict(ht=2), 3), (dict(dt=0, ht=1), 3), (dict(fl=4), 5), (dict(eps=-1.0), 5), (dict(eps=float("nan")), 5),
    (dict(D=16385, gs=1 << 20), 4), (dict(n=1 << 31), 4), (dict(fl=1), 5), (dict(fl=2), 5), (dict(gs=15), 2), (dict(gh=15), 2), (dict(y=None), 1), (dict(h=None), 1), (dict(o=None), 1), (dict(h=0x3000), 6),
    (dict(o=0x6000), 6), (dict(o=0x1000), 6), (dict(y=0x1001), 5), (dict(ht=0, r=0x3002), 5), (dict(n=0, y=None, h=None), 0)])
def test_norm_refusals(lib, kw, status):
    assert _norm(lib, **kw) == status


def _norm_bwd(lib, y=0x1000, g=0x2000, gs=32, gh=16, dt=1, h=0x3000, ht=1, wa=0x4000, wb=0x5000, n=64, heads=2, D=16, eps=1e-6, fl=3, dh=0x6000, dn=0x7000, dy=0x8000, dg=0x9000, dr=0xa000,
              dwa=0xb000, dwb=0xc000, ws=0xd000, wsz=1 << 20):
    return lib.kda_block_norm_bwd(y, g, gs, gh, dt, h, ht, wa, wb, n, heads, D, 1.0, eps, fl, dh, dn, dy, dg, dr, dwa, dwb, ws, wsz, None)


@pytest.mark.parametrize("kw,status", [
    (dict(D=-1), 2), (dict(fl=16), 5), (dict(fl=1, wb=None), 5), (dict(h=None), 1), (dict(dn=None), 1), (dict(dy=None), 1), (dict(dg=None), 1), (dict(ws=None), 1),
    (dict(fl=1, wb=None, dwb=None, dh=None), 1), (dict(dy=0x6000), 6), (dict(dwb=0xb000), 6), (dict(dr=0x3000), 6), (dict(dn=0x7001), 5), (dict(ws=0xd008), 5)])
def test_norm_bwd_refusals(lib, kw, status):
    assert _norm_bwd(lib, **kw) == status


def _steps(lib, which, x=0x1000, dt=1, st=0x6000, pool=8, slots=0x900, cols=3, start=None, lens=None, B=2, S=3, out=0x7000, D=32, W=4):
    if which == "conv":
        return lib.kda_short_conv_step(x, dt, 0x2000, 0x3000, st, pool, slots, cols, start, lens, B, S, D, W, 8, out, None)
    return lib.kda_glr_step(x, dt, 0x2000, 0x3000, 0x4000, -5.0, 0x5000, 1, st, pool, slots, cols, start, lens, B, S, 1, D, out, None)


@pytest.mark.parametrize("which", ["conv", "glr"])
@pytest.mark.parametrize("kw,status", [
    (dict(S=-1), 2), (dict(B=-1), 2), (dict(pool=-1), 2), (dict(D=0), 2), (dict(dt=4), 3), (dict(cols=2), 2), (dict(slots=None), 5), (dict(slots=None, cols=1, pool=1), 5),
    (dict(cols=1, start=0x800), 5), (dict(x=None), 1), (dict(st=None), 1), (dict(out=None), 1), (dict(out=0x1000), 6), (dict(out=0x6000), 6), (dict(st=0x900), 6), (dict(x=0x1001), 5),
    (dict(B=1 << 30), 4), (dict(B=0, x=None), 0), (dict(S=0, x=None), 0)])
def test_step_refusals(lib, which, kw, status):
    assert _steps(lib, which, **kw) == status


def test_where_sequences_begin(tmp_path):
    """The device's own lookup of sequences and their bounds, compiled for the host."""
    exe = str(tmp_path / "rows")
    here = os.path.dirname(os.path.abspath(__file__))
    subprocess.run([HIPCC, "--offload-host-only", "-O1", "-std=c++17", os.path.join(here, "layer_rows_check.hip"), "-o", exe], check=True, capture_output=True, timeout=300)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout


def test_workspace_of_a_single_tile():
    """A shape that is served has a workspace to ask for, the smallest among them."""
    for T in (1, 16, 17):
        for logits in (True, False):
            assert kda.glr_fwd_workspace_size(1, T, 1, 8) > 0 and kda.glr_bwd_workspace_size(1, T, 1, 8, logits, True) > 0
            assert kda.glr_bwd_workspace_size(1, T, 1, 8, logits, False) > 0


def test_python_binding_refuses_cpu_tensors():
    z, w = torch.zeros(1, 4, 2, 16), torch.zeros(32, 4)
    for call in (lambda: kda.short_conv_fwd(z.flatten(2), w), lambda: kda.short_conv_step(z.flatten(2), w, torch.zeros(1, 3, 32)), lambda: kda.glr_fwd(z, z),
                 lambda: kda.glr_step(z, z, torch.zeros(1, 2, 16)), lambda: kda.block_norm_fwd(z), lambda: kda.gated_norm(z), lambda: kda.short_conv_bwd(z.flatten(2), w, z.flatten(2)),
                 lambda: kda.glr_bwd(z, z, z), lambda: kda.block_norm_bwd(z, z, z, z)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        kda.glr_fwd(None, z)


@pytest.mark.parametrize("make,stride", [
    (lambda b: b[:, :, 8:24], 40), (lambda b: b[:1, :, :16], 40), (lambda b: b[:, :1, 3:19], 200), (lambda b: b[:, :, ::2], None), (lambda b: b[:, ::2, :16], None), (lambda b: b[:1, ::2, :16], 80),
    (lambda b: b[:, :3, :16], None), (lambda b: b.transpose(0, 1)[:, :, :16], None), (lambda b: b[:, :, :1].expand(3, 5, 16), None)])
def test_rows_of_a_wider_tensor(make, stride, monkeypatch):
    """A slice whose rows lie at one distance is taken as it is, anything else copied; either way the rows are the same."""
    import gated_delta_rule_31_amd.layer as layer
    monkeypatch.setattr(layer, "_input", lambda x, *a: x.contiguous())
    x = make(torch.arange(600.0).reshape(3, 5, 40))
    got, n = _rows(x, "x")
    width = x.shape[2]
    assert n == (stride or width) and (got.data_ptr() == x.data_ptr()) == (stride is not None)
    flat = torch.as_strided(got, (x.shape[0] * x.shape[1], width), (n, 1), got.storage_offset())
    assert torch.equal(flat, x.reshape(-1, width))


@pytest.mark.parametrize("make,stride,head", [
    (lambda b: b[..., 8:24].unflatten(-1, (2, 8)), 40, 8), (lambda b: b[..., ::2].unflatten(-1, (4, 5)), None, None), (lambda b: b[:, :3, :16].unflatten(-1, (2, 8)), None, None),
    (lambda b: b[..., :20].unflatten(-1, (2, 10))[..., :8], 40, 10), (lambda b: b[1:2, :, 1:17].unflatten(-1, (1, 16)), 40, 16), (lambda b: b[:, 0, 4:12], 200, 8),
    (lambda b: b[..., 4:12], 200, 40), (lambda b: b[0].unflatten(-1, (8, 5)).transpose(0, 1), 5, 40), (lambda b: b[:, :, :1].expand(3, 5, 8), None, None)])
def test_gate_of_a_wider_tensor(make, stride, head, monkeypatch):
    import gated_delta_rule_31_amd.layer as layer
    monkeypatch.setattr(layer, "_input", lambda x, *a: x.contiguous())
    g = make(torch.arange(600.0).reshape(3, 5, 40))
    tokens, heads = layer._tokens_heads(g.shape)
    got, n, h = _gate_rows(g, g, tokens, heads)
    D = g.shape[-1]
    assert (n, h) == ((stride, head) if stride else (heads * D, D)) and (got.data_ptr() == g.data_ptr()) == (stride is not None)
    assert torch.equal(torch.as_strided(got, (tokens, heads, D), (n, h, 1), got.storage_offset()), g.reshape(tokens, heads, D))


def test_reference_gradients():
    """The 64-bit forms' own gradients (automatic differentiation) against differences."""
    gen = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64).requires_grad_()  # noqa: E731
    lens = [3, 0, 1]
    assert torch.autograd.gradcheck(lambda x, w, b, s: ref.conv(x, w, b, s, lens, True), (r(1, 4, 2), r(2, 3), r(2), r(3, 2, 2)))
    assert torch.autograd.gradcheck(lambda x, z, a, b, i, s: ref.scan(x, z, a, b, i, s, lens, True), (r(1, 4, 2, 2), r(1, 4, 2, 2), r(2), r(2, 2), r(1, 4, 2, 2), r(3, 2, 2)))
    assert torch.autograd.gradcheck(lambda y, z, x, a, b: ref.block_norm(y, z, x, a, b, True, True, 0.5, 1e-6, True), (r(2, 5), r(2, 5), r(2, 5), r(5), r(5)))


def test_stretches_of_tiles_keep_their_beginnings(tmp_path):
    """The device's own joining of tiles, in the order of its pass over them, compiled for the host."""
    exe = str(tmp_path / "carry")
    here = os.path.dirname(os.path.abspath(__file__))
    subprocess.run([HIPCC, "--offload-host-only", "-O1", "-std=c++17", os.path.join(here, "layer_carry_check.hip"), "-o", exe], check=True, capture_output=True, timeout=300)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout


# Float32 and int32 pointers off a 4-byte border, in calls with rows and without
FLOATS = {
    "conv": (_conv, dict(w=0x2002, b=0x3001, cu=0x902), dict(T=0)), "conv_states": (_conv, dict(s0=0x9002, sf=0xa002), dict(T=0)),
    "conv_bwd": (_conv_bwd, dict(w=0x2002, b=0x3002, cu=0x901, dw=0x6002, db=0x7002), dict(T=0)),
    "conv_bwd_states": (_conv_bwd, dict(s0=0x9002, dsf=0xa002, ds0=0xb002), dict(T=0)),
    "glr": (_glr, dict(ls=0x3002, b=0x4001, s0=0x9002, sf=0xa002, cu=0x902, kept=0xb002), dict(T=0)),
    "glr_bwd": (_glr_bwd, dict(ls=0x3002, b=0x4002, s0=0x9002, cu=0x902, kept=0x6002, dsf=0xe002, dls=0xb002, db=0xc002, ds0=0xf002), dict(T=0)),
    "norm": (_norm, dict(wa=0x4002, wb=0x5001), dict(n=0)), "norm_bwd": (_norm_bwd, dict(wa=0x4002, wb=0x5002, dwa=0xb002, dwb=0xc001), dict(n=0))}


@pytest.mark.parametrize("call,name", [(c, n) for c in FLOATS for n in FLOATS[c][1]])
def test_float_pointers_off_a_border(lib, call, name):
    fn, off, empty = FLOATS[call]
    kw = {name: off[name]}
    if name == "cu":
        kw["N"] = 1
    if call.endswith("states"):
        kw["dt"] = 0
    assert fn(lib, **kw) == 5 and fn(lib, **kw, **empty) == 5


@pytest.mark.parametrize("which", ["conv", "glr"])
@pytest.mark.parametrize("kw", [dict(slots=0x902), dict(start=0x802), dict(lens=0x801), dict(st=0x6002, dt=0)])
def test_step_pointers_off_a_border(lib, which, kw):
    assert _steps(lib, which, **kw) == 5


@pytest.mark.parametrize("kw", [dict(ls=0x3002), dict(b=0x4002), dict(st=0x6002)])
def test_glr_step_pointers_off_a_border(lib, kw):
    arg = dict(ls=0x3000, b=0x4000, st=0x6000)
    arg.update(kw)
    assert lib.kda_glr_step(0x1000, 1, 0x2000, arg["ls"], arg["b"], -5.0, 0x5000, 1, arg["st"], 8, 0x900, 3, None, None, 2, 3, 1, 32, 0x7000, None) == 5


@pytest.mark.parametrize("w,b", [(0x2002, 0x3000), (0x2000, 0x3002)])
def test_conv_step_pointers_off_a_border(lib, w, b):
    assert lib.kda_short_conv_step(0x1000, 1, w, b, 0x6000, 8, 0x900, 3, None, None, 2, 3, 32, 4, 8, 0x7000, None) == 5


def test_forward_mode_is_refused():
    """A dual tensor that does not require grad is refused by every call that would drop its tangent, also without grad mode;
    outside of its level it is an ordinary tensor."""
    from torch.autograd import forward_ad
    plain, w = torch.zeros(1, 4, 2, 16), torch.zeros(32, 4)
    dual = lambda t: forward_ad.make_dual(t, torch.ones_like(t))  # noqa: E731
    with forward_ad.dual_level():
        z = dual(plain)
        calls = [lambda: kda.short_conv(z.flatten(2), w), lambda: kda.short_conv_fwd(z.flatten(2)[..., 8:24], w), lambda: kda.short_conv_step(z.flatten(2), w, torch.zeros(1, 3, 32)),
                 lambda: kda.gated_linear_recurrence(z, plain), lambda: kda.glr_fwd(z, plain), lambda: kda.glr_step(z, plain, torch.zeros(1, 2, 16)), lambda: kda.block_norm(z),
                 lambda: kda.block_norm_fwd(z), lambda: kda.gated_norm(z), lambda: kda.short_conv_bwd(z.flatten(2), w, plain.flatten(2)), lambda: kda.glr_bwd(z, plain, plain),
                 lambda: kda.block_norm_bwd(z, plain, plain, plain), lambda: kda.gdr_chunk_fwd(z, plain, plain, plain[..., 0], plain[..., 0]),
                 lambda: kda.gated_delta_rule(z, plain, plain, plain[..., 0], plain[..., 0]), lambda: kda.bounded_decay(z, torch.zeros(2)),
                 lambda: kda.chunk_fwd(z, plain, plain, plain, plain[..., 0]), lambda: kda.recurrent_fwd(z, plain, plain, plain, plain[..., 0])]
        for grad in (True, False):
            with torch.set_grad_enabled(grad):
                for call in calls:
                    with pytest.raises(ValueError, match="forward-mode tangent"):
                        call()
        for call in (lambda: kda.short_conv_fwd(plain.flatten(2), w), lambda: kda.bounded_decay(plain, torch.zeros(2))):
            with pytest.raises(ValueError, match="on the GPU"):
                call()
    with pytest.raises(ValueError, match="on the GPU"):
        kda.glr_fwd(z, plain)


def test_many_sequences_without_rows(tmp_path):
    """The device's own lookup of where sequences begin, compiled for the host, in batches padded with up to 2^20 empty sequences."""
    exe = str(tmp_path / "empty")
    here = os.path.dirname(os.path.abspath(__file__))
    subprocess.run([HIPCC, "--offload-host-only", "-O1", "-std=c++17", os.path.join(here, "layer_empty_check.hip"), "-o", exe], check=True, capture_output=True, timeout=300)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout
