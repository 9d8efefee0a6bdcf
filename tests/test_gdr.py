"""CPU checks of the gated delta rule's C entry points: refusals before any launch (the
pointers are fake), workspace sizes, and the Python binding's checks."""
import ctypes
import os

import pytest
import torch

import gated_delta_rule_31_amd as kda

vp, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t


@pytest.fixture(scope="module")
def lib():
    assert os.path.exists(kda.library_path()), "libkda.so is not built"
    return kda._load()


def _fwd(lib, q=0x1000, k=0x2000, v=0x3000, dt=1, g=0x4000, beta=0x5000, s0=None, sf=None, cu=None, N=0, B=1, T=64, HK=2, HV=4, K=16, V=16,
         out=0x6000, od=1, ws=0x7000, wsz=1 << 24):
    return lib.kda_gdr_chunk_fwd(q, k, v, dt, g, beta, s0, sf, cu, N, B, T, HK, HV, K, V, 1.0, out, od, ws, wsz, None)


@pytest.mark.parametrize("kw,status", [
    (dict(K=24), 4), (dict(V=256), 4), (dict(HK=0), 2), (dict(HV=3), 2), (dict(HK=4, HV=2), 2), (dict(T=-1), 2), (dict(B=-1), 2),
    (dict(dt=5), 3), (dict(od=7), 3), (dict(q=None), 1), (dict(g=None), 1), (dict(out=None), 1), (dict(ws=None), 1),
    (dict(cu=0x900, B=2, N=2), 5), (dict(cu=0x900, N=-1), 5), (dict(cu=0x900, N=0), 5), (dict(HK=1, HV=65536), 4), (dict(B=1 << 22), 4), (dict(out=0x1000), 6), (dict(sf=0x3000), 6), (dict(ws=0x1000), 6),
    (dict(sf=0x6000), 6), (dict(ws=0x6000), 6), (dict(q=0x1004), 5), (dict(out=0x6008), 5), (dict(ws=0x7004), 5), (dict(s0=0x8004), 5),
    (dict(wsz=64), 5), (dict(T=1 << 40), 4),
    (dict(T=0, q=None, out=None, ws=None), 0), (dict(B=0, q=None, out=None, ws=None), 0),
])
def test_chunk_fwd_refusals(lib, kw, status):
    assert _fwd(lib, **kw) == status


def test_chunk_fwd_workspace(lib):
    size = lambda dt=torch.bfloat16, B=1, T=64, HK=2, HV=4, K=16, V=16, N=0, packed=False: kda.gdr_chunk_fwd_workspace_size(  # noqa: E731
        dt, B, T, HK, HV, K, V, N, packed)
    # three bf16 parts of M and two of P (three with float32 inputs), and four rows of 64 floats
    assert size() == 4 * ((3 + 2) * 64 * 64 * 2 + 4 * 64 * 4) and size(torch.float32) == 4 * ((3 + 3) * 64 * 64 * 2 + 4 * 64 * 4)
    assert size(T=65) == 2 * size() == size(B=2) and size(T=64 * 7) == 7 * size()
    assert size(T=130, N=4, packed=True) == 6 * size()  # T // 64 + N chunk slots
    assert size(K=24) == 0 and size(HV=3) == 0 and size(T=0) == 0
    need = size()
    assert _fwd(lib, wsz=need - 1) == 5


def _bwd(lib, q=0x1000, k=0x2000, v=0x3000, dt=1, g=0x4000, beta=0x5000, s0=None, cu=None, N=0, B=1, T=64, HK=2, HV=4, K=16, V=16, do=0x6000,
         dd=1, dsf=None, dq=0x7000, dk=0x8000, dv=0x9000, gd=1, dg=0xa000, db=0xb000, ds0=None, ws=0xc000, wsz=1 << 30):
    return lib.kda_gdr_chunk_bwd(q, k, v, dt, g, beta, s0, cu, N, B, T, HK, HV, K, V, 1.0, do, dd, dsf, dq, dk, dv, gd, dg, db, ds0, ws, wsz,
                                 None)


@pytest.mark.parametrize("kw,status", [
    (dict(K=8), 4), (dict(HV=5), 2), (dict(dt=4), 3), (dict(dd=4), 3), (dict(gd=4), 3), (dict(do=None), 1), (dict(dg=None), 1), (dict(ws=None), 1),
    (dict(cu=0x900, B=2), 5), (dict(dq=0x2000), 6), (dict(dg=0x7000), 6), (dict(ds0=0x6000), 6), (dict(ws=0x6000), 6), (dict(do=0x6008), 5),
    (dict(wsz=4096), 5), (dict(T=0, q=None, ws=None), 0),
])
def test_chunk_bwd_refusals(lib, kw, status):
    assert _bwd(lib, **kw) == status


def test_chunk_bwd_workspace(lib):
    size = lambda **kw: kda.gdr_chunk_bwd_workspace_size(**{**dict(dtype=torch.bfloat16, B=1, T=64, HK=2, HV=4, K=16, V=32), **kw})  # noqa: E731
    # three bf16 parts of M, M^T and P^T; decays (float) and their sums (double); two states and two sets of rows; with
    # float32 inputs three parts of K^T and Q^T for a key head
    assert size() == 4 * (3 * 3 * 64 * 64 * 2 + 4 * 64 * 4 + 64 * 8 + 2 * 16 * 32 * 4 + 2 * 64 * 32 * 4)
    assert size(dtype=torch.float32) == size() + 2 * 2 * 3 * 16 * 64 * 2
    assert size(T=130, num_seqs=4, varlen=True) == 6 * size() and size(K=24) == 0 and size(T=0, num_seqs=3, varlen=True) == 0
    assert _bwd(lib, V=32, wsz=size() - 1) == 5


def _step(lib, q=0x1000, k=0x2000, v=0x3000, dt=1, g=0x4000, ch=0, beta=0x5000, st=0x6000, pool=8, slots=0x900, cols=3, start=None, lens=None,
          B=2, S=3, HK=2, HV=4, K=16, V=16, out=0x7000, od=1):
    return lib.kda_gdr_recurrent_step(q, k, v, dt, g, ch, beta, st, pool, slots, cols, start, lens, B, S, HK, HV, K, V, 1.0, out, od, None)


@pytest.mark.parametrize("kw,status", [
    (dict(K=48), 4), (dict(HV=5), 2), (dict(S=-1), 2), (dict(pool=-1), 2), (dict(dt=3), 3), (dict(od=3), 3), (dict(cols=2), 2),
    (dict(slots=None, cols=3), 5), (dict(slots=None, cols=1, start=0x800), 5), (dict(slots=None, cols=1, pool=1), 5), (dict(cols=1, start=0x800), 5),
    (dict(st=None), 1), (dict(beta=None), 1), (dict(out=None), 1), (dict(out=0x3000), 6), (dict(st=0x1000), 6), (dict(out=0x6000), 6),
    (dict(st=0x6004), 5), (dict(g=0x4004, ch=1), 5), (dict(B=1 << 30), 4), (dict(B=0, q=None, st=None), 0), (dict(S=0, q=None, st=None), 0),
])
def test_step_refusals(lib, kw, status):
    assert _step(lib, **kw) == status


def _verify(lib, p=0x1000, x=0x2000, q=0x3000, u=0x4000, lens=None, B=2, D=3, vocab=100, t=0x5000, a=0x6000, ws=0x7000, wsz=1 << 20):
    return lib.kda_draft_verify(p, x, q, u, lens, B, D, vocab, t, a, ws, wsz, None)


@pytest.mark.parametrize("kw,status", [
    (dict(D=-1), 2), (dict(vocab=0), 2), (dict(vocab=(1 << 19) + 1), 4), (dict(B=1 << 30), 4), (dict(p=None), 1), (dict(x=None), 1),
    (dict(u=None), 1), (dict(t=None), 1), (dict(ws=None), 1), (dict(t=0x2000), 6), (dict(a=0x5000), 6), (dict(ws=0x1000), 6),
    (dict(ws=0x7004), 5), (dict(wsz=31), 5), (dict(B=1 << 20, vocab=1 << 19), 4), (dict(B=0, p=None), 0),
])
def test_verify_refusals(lib, kw, status):
    assert _verify(lib, **kw) == status


def test_python_binding_refuses_cpu_tensors():
    z = torch.zeros(1, 4, 2, 16)
    with pytest.raises(ValueError):
        kda.gdr_chunk_fwd(z, z, z, z[..., 0], z[..., 0])
    with pytest.raises(ValueError):
        kda.gdr_recurrent_step(z, z, z, z[..., 0], z[..., 0], torch.zeros(1, 2, 16, 16))
    with pytest.raises(ValueError):
        kda.draft_verify(torch.zeros(1, 2, 5), torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, 2))
