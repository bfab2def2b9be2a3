"""The layer operators refuse bad host arguments before anything is launched
(CPU only: stand-in addresses, no call here reaches a kernel launch)."""
from __future__ import annotations

import ctypes
import os

import pytest
import torch

import depthwise_causal_conv1d_amd as sc


@pytest.fixture(scope="module")
def lib():
    from depthwise_causal_conv1d_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        from depthwise_causal_conv1d_amd import build
        build.build()
    return _lib.load()


MB = 1 << 20
# far-apart stand-in addresses
X, GA, GX, OUT, ST, MK, DO, DX, DGA, DGX, DEC, DD, WS, QSL, IDX, HAS, DF, DI = (
    (1 << 40) + k * 64 * MB for k in range(18))


def err(lib):
    return lib.sconv_last_error().decode()


def fwd(lib, **kw):
    a = dict(x=X, xc=64, xt=1, ga=GA, gac=64, gat=1, gx=GX, gxc=64, gxt=1, decay=DEC, scale=8.0,
             st=ST, slots=4, ss=16, qsl=QSL, batch=2, idx=IDX, has=HAS, out=OUT, oc=64, ot=1,
             mk=MK, rows=4, ws=None, wsn=0, dim=16, T=64, dt=0, pad=-1)
    a.update(kw)
    return lib.gated_linear_recurrence_varlen_fwd(*a.values(), None)


@pytest.mark.parametrize("kw,text", [
    (dict(batch=-1), ">= 0"), (dict(dim=-1), ">= 0"), (dict(T=-1), ">= 0"), (dict(dt=2), "dtype"),
    (dict(dt=9), "dtype"), (dict(scale=0.0), "decay_scale"), (dict(scale=-1.0), "decay_scale"),
    (dict(scale=float("nan")), "decay_scale"), (dict(scale=float("inf")), "decay_scale"),
    (dict(x=None), "NULL"), (dict(ga=None), "NULL"), (dict(gx=None), "NULL"),
    (dict(out=None), "NULL"), (dict(decay=None), "NULL"), (dict(qsl=None), "NULL"),
    (dict(st=None), "without states"), (dict(slots=0), "slots"),
    (dict(idx=None, slots=1), "slots"), (dict(ss=15), "slot stride"), (dict(rows=3), "checkpoints"),
    (dict(xc=-1), "strides"), (dict(gat=-1), "strides"), (dict(oc=0), "each other"),
    (dict(oc=63), "each other"), (dict(out=X + 4), "overlaps x"), (dict(out=X, oc=65), "overlaps x"),
    (dict(out=GA), "gate"), (dict(out=GX), "gate"), (dict(st=OUT), "overlap"),
    (dict(mk=OUT + 64), "overlap"), (dict(mk=ST), "overlap"), (dict(st=X + 4092), "overlap"),
])
def test_recurrence_forward_refusals(lib, kw, text):
    assert fwd(lib, **kw) == 1 and text in err(lib), err(lib)


def test_recurrence_forward_workspace_refusals(lib):
    """One sequence of 65536 tokens in rows: cut over its tokens."""
    fwd_n, bwd_n = ctypes.c_int64(), ctypes.c_int64()
    f = lib.gated_linear_recurrence_workspace
    assert f(65536, 1, 16, ctypes.byref(fwd_n), ctypes.byref(bwd_n)) == 0
    assert fwd_n.value > 0 and bwd_n.value > fwd_n.value
    kw = dict(xc=1, xt=16, gac=1, gat=16, gxc=1, gxt=16, oc=1, ot=16, batch=1, T=65536, rows=2049)
    assert fwd(lib, **kw, ws=WS, wsn=fwd_n.value - 1) == 1 and "workspace holds" in err(lib)
    assert fwd(lib, **kw, ws=X + 64, wsn=fwd_n.value) == 1 and "workspace overlaps" in err(lib)
    assert fwd(lib, **kw, ws=MK, wsn=fwd_n.value) == 1 and "workspace overlaps" in err(lib)
    for bad in ((-1, 1, 1), (1, -1, 1), (1, 1, -1)):
        assert f(*bad, ctypes.byref(fwd_n), ctypes.byref(bwd_n)) == 1
    assert f(1, 1, 1, None, ctypes.byref(bwd_n)) == 1 and f(1, 1, 1, ctypes.byref(fwd_n), None) == 1


def test_recurrence_forward_no_ops_and_limits(lib):
    assert fwd(lib, batch=0) == 0 and fwd(lib, dim=0) == 0
    # more threads than one launch takes, whatever the kernel
    assert fwd(lib, batch=1 << 30, dim=1 << 14, T=1, st=None, has=None, mk=None) == 2
    # token numbers are int32, a channel's byte offset in a row 32 bits
    assert fwd(lib, T=(1 << 31) - 4096) == 2 and bwd(lib, T=(1 << 31) - 4096) == 2
    assert fwd(lib, dim=(1 << 28) + 1) == 2 and cgrad(lib, dim=(1 << 28) + 1) == 2
    assert cgrad(lib, T=(1 << 31) - 4096) == 2


def bwd(lib, **kw):
    a = dict(do=DO, doc=64, dot=1, x=X, xc=64, xt=1, ga=GA, gac=64, gat=1, gx=GX, gxc=64, gxt=1,
             decay=DEC, scale=8.0, mk=MK, rows=4, qsl=QSL, batch=2, idx=IDX, has=HAS, slots=4,
             df=DF, dfs=16, di=DI, dis=16, dx=DX, dxc=64, dxt=1, dga=DGA, dgac=64, dgat=1, dgx=DGX,
             dgxc=64, dgxt=1, dd=DD, ws=WS, wsn=32, dim=16, T=64, dt=0, pad=-1)
    a.update(kw)
    return lib.gated_linear_recurrence_varlen_bwd(*a.values(), None)


@pytest.mark.parametrize("kw,text", [
    (dict(batch=-1), ">= 0"), (dict(dt=5), "dtype"), (dict(scale=0.0), "decay_scale"),
    (dict(do=None), "NULL"), (dict(mk=None), "NULL"), (dict(dd=None), "NULL"),
    (dict(ws=None), "NULL"), (dict(dga=None), "NULL"), (dict(rows=3), "checkpoints"),
    (dict(wsn=31), "workspace"), (dict(slots=0), "slots"), (dict(idx=None, slots=1), "slots"),
    (dict(dfs=8), "slot stride"), (dict(dis=8), "slot stride"), (dict(doc=-1), "strides"),
    (dict(dxt=0), "each other"), (dict(dx=X), "overlaps an input"), (dict(dx=DO), "overlaps an input"),
    (dict(dgx=DGA), "two gradients"), (dict(dx=MK), "overlaps an input"),
    (dict(dx=DF), "overlaps an input"), (dict(di=DF + 64), "overlap another"),
    (dict(di=DF, dis=32), "overlap another"), (dict(dd=X), "overlap another"),
    (dict(ws=MK), "overlap another"), (dict(ws=DD), "overlap another"), (dict(dd=DEC), "overlap another"),
])
def test_recurrence_backward_refusals(lib, kw, text):
    assert bwd(lib, **kw) == 1 and text in err(lib), err(lib)


def test_recurrence_checkpoint_rows(lib):
    n = ctypes.c_int64()
    f = lib.gated_linear_recurrence_checkpoint_rows
    for T, b, want in ((0, 0, 0), (0, 3, 3), (1, 1, 2), (32, 1, 2), (33, 2, 4)):
        assert f(T, b, ctypes.byref(n)) == 0 and n.value == want
    assert f(-1, 1, ctypes.byref(n)) == 1 and f(1, -1, ctypes.byref(n)) == 1 and f(1, 1, None) == 1


def upd(lib, **kw):
    a = dict(x=X, xb=16, ga=GA, gab=16, gx=GX, gxb=16, decay=DEC, scale=8.0, st=ST, slots=4, ss=16,
             idx=IDX, out=OUT, ob=16, batch=2, dim=16, dt=1, pad=-1)
    a.update(kw)
    return lib.gated_linear_recurrence_update(*a.values(), None)


@pytest.mark.parametrize("kw,text", [
    (dict(batch=-1), ">= 0"), (dict(dim=-1), ">= 0"), (dict(dt=2), "dtype"), (dict(scale=0.0), "decay_scale"),
    (dict(x=None), "NULL"), (dict(st=None), "NULL"), (dict(out=None), "NULL"),
    (dict(slots=0), "slots"), (dict(idx=None, slots=1), "slots"), (dict(ss=8), "slot stride"),
    (dict(xb=-1), "strides"), (dict(ob=15), "each other"), (dict(out=X + 2), "overlaps x"),
    (dict(out=GA), "gate"), (dict(st=OUT), "overlap"),
])
def test_recurrence_update_refusals(lib, kw, text):
    assert upd(lib, **kw) == 1 and text in err(lib), err(lib)


def test_recurrence_update_no_ops(lib):
    assert upd(lib, batch=0) == 0 and upd(lib, dim=0) == 0


def cgrad(lib, **kw):
    a = dict(do=DO, doc=64, dot=1, x=X, xc=64, xt=1, w=DEC, wc=4, wk=1, bias=GA, ini=ST, iss=48,
             isc=3, isk=1, slots=4, qsl=QSL, batch=2, idx=IDX, has=HAS, df=DF, dfs=48, dfc=3, dfk=1,
             di=DI, dis=48, dic=3, dik=1, dx=DX, dxc=64, dxt=1, dw=DGA, db=DGX, ws=WS, wsn=160,
             dim=16, T=64, W=4, dt=0, act=1, pad=-1)
    a.update(kw)
    return lib.causal_conv1d_varlen_bwd(*a.values(), None)


@pytest.mark.parametrize("kw,text", [
    (dict(T=-1), ">= 0"), (dict(W=0), "W=0"), (dict(W=5), "W=5"), (dict(dt=2), "dtype"),
    (dict(act=2), "activation"), (dict(do=None), "NULL"), (dict(dx=None), "NULL"),
    (dict(dw=None), "NULL"), (dict(ws=None), "NULL"), (dict(w=None), "NULL"),
    (dict(ini=None), "without initial_states"), (dict(slots=0), "slots"),
    (dict(idx=None, slots=1), "slots"), (dict(wc=-1), "strides"), (dict(dic=0), "strides"),
    (dict(isk=-1), "strides"), (dict(wsn=159), "workspace"), (dict(xt=-1), "strides"),
    (dict(dxc=10), "each other"), (dict(dx=X), "overlaps dout or x"), (dict(dx=DO), "overlaps dout or x"),
    (dict(dx=ST), "overlaps another"), (dict(di=DF), "overlaps another"),
    (dict(di=ST), "overlaps another"), (dict(dw=DEC), "overlaps another"),
    (dict(db=DGA), "overlaps another"), (dict(ws=X + 64), "overlaps another"),
])
def test_conv_gradient_refusals(lib, kw, text):
    assert cgrad(lib, **kw) == 1 and text in err(lib), err(lib)


def test_conv_gradient_workspace(lib):
    n = ctypes.c_int64()
    f = lib.causal_conv1d_varlen_bwd_workspace
    assert f(64, 2, 16, 4, ctypes.byref(n)) == 0 and n.value >= 2 * 16 * 5
    assert f(64, 0, 16, 4, ctypes.byref(n)) == 0 and n.value == 0
    for bad in ((-1, 1, 1, 4), (1, -1, 1, 4), (1, 1, -1, 4), (1, 1, 1, 0), (1, 1, 1, 5)):
        assert f(*bad, ctypes.byref(n)) == 1
    assert f(1, 1, 1, 4, None) == 1


def norm(lib, **kw):
    a = dict(x=X, xr=256, res=GA, rr=256, w=DEC, eps=1e-6, so=GX, sr=256, out=OUT, orr=256, sc=ST,
             scr=2, group=128, rows=4, dim=256, dt=1, odt=2)
    a.update(kw)
    return lib.rms_norm_fwd(*a.values(), None)


@pytest.mark.parametrize("kw,rc,text", [
    (dict(rows=-1), 1, ">= 0"), (dict(dt=2), 1, "dtype"), (dict(odt=0), 1, "out_dtype"),
    (dict(odt=1), 1, "group_size"), (dict(eps=-1.0), 1, "eps"), (dict(eps=float("nan")), 1, "eps"),
    (dict(group=-1), 1, "group_size"), (dict(group=100), 2, "none of"), (dict(group=512, dim=1024), 2, "none of"),
    (dict(dim=200), 1, "divide"), (dict(x=None), 1, "NULL"), (dict(w=None), 1, "NULL"),
    (dict(out=None), 1, "NULL"), (dict(sc=None), 1, "NULL"), (dict(res=None), 1, "without residual"),
    (dict(xr=-1), 1, "strides"), (dict(sr=255), 1, "each other"), (dict(orr=200), 1, "each other"),
    (dict(scr=1), 1, "each other"), (dict(out=X), 1, "partially"), (dict(so=X + 2), 1, "partially"),
    (dict(so=GA, sr=260), 1, "partially"), (dict(out=GX), 1, "two outputs"), (dict(sc=OUT), 1, "two outputs"),
    (dict(sc=GA), 1, "partially"), (dict(so=DEC), 1, "weight"),
])
def test_norm_refusals(lib, kw, rc, text):
    assert norm(lib, **kw) == rc and text in err(lib), err(lib)


def nbwd(lib, **kw):
    a = dict(do=DO, dor=256, x=X, xr=256, w=DEC, eps=1e-6, dr=GA, drr=256, dx=DX, dxr=256, dw=DGA,
             ws=WS, wsn=1 << 22, rows=4, dim=256, dt=1)
    a.update(kw)
    return lib.rms_norm_bwd(*a.values(), None)


@pytest.mark.parametrize("kw,text", [
    (dict(rows=-1), ">= 0"), (dict(dt=2), "dtype"), (dict(eps=-1.0), "eps"), (dict(do=None), "NULL"),
    (dict(dx=None), "NULL"), (dict(dw=None), "NULL"), (dict(ws=None), "NULL"), (dict(wsn=0), "workspace"),
    (dict(xr=-1), "strides"), (dict(dxr=255), "each other"), (dict(dx=X + 2), "partially"),
    (dict(dx=DO, dxr=300), "partially"), (dict(dw=X), "overlaps another"),
    (dict(dw=WS), "overlaps another"), (dict(dx=DEC), "overlaps another"),
])
def test_norm_backward_refusals(lib, kw, text):
    assert nbwd(lib, **kw) == 1 and text in err(lib), err(lib)


def test_norm_no_ops_and_workspace(lib):
    assert norm(lib, rows=0) == 0 and norm(lib, dim=0) == 0 and nbwd(lib, dim=0) == 0
    n = ctypes.c_int64()
    assert lib.rms_norm_bwd_workspace(0, 8, ctypes.byref(n)) == 0 and n.value == 0
    assert lib.rms_norm_bwd_workspace(7, 8, ctypes.byref(n)) == 0 and n.value > 0
    assert lib.rms_norm_bwd_workspace(-1, 8, ctypes.byref(n)) == 1
    assert lib.rms_norm_bwd_workspace(1, 8, None) == 1


# ---------------------------------------------------------------- the binding

def test_binding_wants_gpu_tensors_of_one_type_and_shape():
    x, d = torch.zeros(4, 8), torch.zeros(4)
    q = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        sc.gated_linear_recurrence_varlen_fwd(x, x, x, d, None, q)
    with pytest.raises(ValueError, match="GPU"):
        sc.gated_linear_recurrence_varlen_bwd(x, x, x, x, d, x, q)
    with pytest.raises(ValueError, match="GPU"):
        sc.gated_linear_recurrence_update(x, x, x, torch.zeros(8), x)
    with pytest.raises(ValueError, match="GPU"):
        sc.causal_conv1d_varlen_bwd(x, x, torch.zeros(4, 4), None, None, q, None, None, True)
    for f in (sc.rms_norm_fwd, sc.rms_norm_quant):
        with pytest.raises(ValueError, match="GPU"):
            f(x, torch.zeros(8))
    with pytest.raises(ValueError, match="GPU"):
        sc.rms_norm_bwd(x, x, torch.zeros(8))
    with pytest.raises(ValueError, match=r"\[dim, total_T\]"):
        sc.gated_linear_recurrence_varlen_fwd(d, d, d, d, None, q)
    with pytest.raises(ValueError, match="divide"):
        sc.rms_norm_quant(x, torch.zeros(8), group_size=3)
    with pytest.raises(TypeError):
        sc.rms_norm_fwd(x, torch.zeros(8), out=torch.zeros(4, 8, dtype=torch.bfloat16))


def test_recurrence_outputs_do_not_overlap_decay(lib):
    """Every channel of every workgroup reads decay while others write."""
    rows = dict(xc=1, xt=16, gac=1, gat=16, gxc=1, gxt=16, oc=1, ot=16, batch=1, T=65536, rows=2049)
    fwd_n, bwd_n = ctypes.c_int64(), ctypes.c_int64()
    assert lib.gated_linear_recurrence_workspace(65536, 1, 16, ctypes.byref(fwd_n),
                                                 ctypes.byref(bwd_n)) == 0
    calls = [lambda: fwd(lib, decay=OUT), lambda: fwd(lib, decay=ST + 60), lambda: fwd(lib, decay=MK),
             lambda: fwd(lib, **rows, decay=WS, ws=WS, wsn=fwd_n.value),
             lambda: upd(lib, decay=OUT + 16), lambda: upd(lib, decay=ST)]
    calls += [lambda k=k: bwd(lib, decay=k) for k in (DX, DGA + 4, DGX, DI, DD, WS)]
    for k, call in enumerate(calls):
        assert call() == 1 and "overlap" in err(lib), (k, err(lib))
