"""The gated delta rule, the layer norm and the paged metadata refuse bad host
arguments before anything is launched (CPU only: stand-in addresses, no call
here reaches a kernel launch)."""
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
Q, K, V, G, B, OUT, ST, MK, WS, QSL, IDX, HAS, DO, DQ, DK, DV, DG, DB, DF, DI = (
    (1 << 40) + n * 64 * MB for n in range(20))
ONE = 2 * 16 * 8  # floats of a slot: 2 value heads, K = 16, V = 8


def err(lib):
    return lib.sconv_last_error().decode()


def inputs():
    return dict(q=Q, qt=16, qh=16, k=K, kt=16, kh=16, v=V, vt=16, vh=8, g=G, gt=2, gh=1, b=B, bt=2, bh=1,
                scale=0.25)


def sizes():
    return dict(T=64, heads_k=1, heads_v=2, K=16, V=8, dt=0, gdt=0, pad=-1)


def fwd(lib, **kw):
    a = inputs() | dict(st=ST, slots=4, ss=ONE, qsl=QSL, batch=2, idx=IDX, has=HAS, out=OUT, ot=16, oh=8, mk=MK,
                        rows=4, ws=WS, wsn=1 << 22) | sizes()
    assert set(kw) <= set(a)
    return lib.gated_delta_rule_varlen_fwd(*(a | kw).values(), None)


SHARED = [
    (dict(batch=-1), "negative"), (dict(T=-1), "negative"), (dict(K=-1), "negative"), (dict(V=-1), "negative"),
    (dict(dt=2), "dtype"), (dict(dt=9), "dtype"), (dict(dt=1, gdt=2), "g and beta"), (dict(dt=0, gdt=1), "g and beta"),
    (dict(heads_v=3, heads_k=2), "evenly"), (dict(heads_k=0), "evenly"), (dict(K=0), "positive"),
    (dict(scale=float("nan")), "scale"), (dict(scale=float("inf")), "scale"),
    (dict(q=None), "NULL"), (dict(k=None), "NULL"), (dict(v=None), "NULL"), (dict(g=None), "NULL"),
    (dict(b=None), "NULL"), (dict(qt=-1), "stride"), (dict(kh=-1), "stride"), (dict(vt=-1), "stride"),
    (dict(gt=-1), "stride"), (dict(bh=-1), "stride"),
]


@pytest.mark.parametrize("kw,text", SHARED + [
    (dict(qsl=None), "NULL"), (dict(out=None), "NULL"), (dict(st=None), "without states"),
    (dict(ss=ONE - 1), "slots overlap"), (dict(idx=None, slots=1), "slots"), (dict(rows=3), "checkpoint"),
    (dict(mk=MK + 4), "16 bytes"), (dict(ws=None), "workspace"), (dict(wsn=100), "workspace"), (dict(ws=WS + 4), "workspace"),
    (dict(ot=15), "share memory"), (dict(oh=7), "share memory"), (dict(ot=0), "share memory"),
    (dict(ot=-1), "stride"), (dict(out=V + 4), "overlaps an input"), (dict(out=V, ot=17), "overlaps an input"),
    (dict(out=Q), "overlaps an input"), (dict(out=K + 64), "overlaps an input"), (dict(out=G), "overlaps an input"),
    (dict(out=B + 8), "overlaps an input"), (dict(st=OUT), "overlap"), (dict(mk=ST + 64), "overlap"),
    (dict(mk=OUT), "overlap"), (dict(ws=MK), "overlap"), (dict(ws=Q), "overlap"), (dict(st=V), "overlap"),
])
def test_forward_refusals(lib, kw, text):
    assert fwd(lib, **kw) == 1 and text in err(lib), err(lib)


def test_no_ops_and_limits(lib):
    assert fwd(lib, batch=0) == 0 and fwd(lib, heads_v=0) == 0 and fwd(lib, V=0) == 0
    for f in (fwd, bwd, upd):
        assert f(lib, K=129) == 2, err(lib)
        assert f(lib, batch=65536) == 2
        assert f(lib, heads_v=1 << 17) == 2
        assert f(lib, V=(1 << 20) + 1) == 2
    assert fwd(lib, T=(1 << 31) - 4096) == 2 and bwd(lib, T=(1 << 31) - 4096) == 2
    assert fwd(lib, T=1 << 30) == 2  # more chunks than one launch takes
    assert fwd(lib, T=3 << 27) == 2 and bwd(lib, T=3 << 27) == 2
    assert bwd(lib, batch=0) == 0 and bwd(lib, V=0) == 0 and upd(lib, batch=0) == 0


def bwd(lib, **kw):
    a = dict(do=DO, dot=16, doh=8) | inputs() | dict(
        mk=MK, rows=4, qsl=QSL, batch=2, idx=IDX, has=HAS, slots=4, df=DF, dfs=ONE, di=DI, dis=ONE, dq=DQ, dqt=16,
        dqh=16, dk=DK, dkt=16, dkh=16, dv=DV, dvt=16, dvh=8, dg=DG, dgt=2, dgh=1, db=DB, dbt=2, dbh=1, ws=WS,
        wsn=1 << 22) | sizes()
    assert set(kw) <= set(a)
    return lib.gated_delta_rule_varlen_bwd(*(a | kw).values(), None)


@pytest.mark.parametrize("kw,text", SHARED + [
    (dict(qsl=None), "NULL"), (dict(do=None), "NULL"), (dict(mk=None), "NULL"), (dict(dot=-1), "stride"),
    (dict(rows=3), "checkpoint"), (dict(mk=MK + 8), "16 bytes"), (dict(dfs=ONE - 1), "slots overlap"), (dict(dis=ONE - 1), "slots overlap"),
    (dict(idx=None, slots=1), "slots"), (dict(dq=None), "NULL"), (dict(dk=None), "NULL"), (dict(dv=None), "NULL"),
    (dict(dg=None), "NULL"), (dict(db=None), "NULL"), (dict(dqt=15), "share memory"), (dict(dvh=7), "share memory"),
    (dict(dgt=1), "share memory"), (dict(dbh=0), "share memory"), (dict(ws=None), "workspace"),
    (dict(wsn=1 << 10), "workspace"), (dict(ws=WS + 8), "workspace"), (dict(di=DF + 64), "overlap"),
    (dict(di=DF, dis=2 * ONE), "overlap"), (dict(dq=MK), "overlaps an input"), (dict(dv=DO), "overlaps an input"),
    (dict(dv=V), "overlaps an input"), (dict(dq=Q), "overlaps an input"), (dict(dq=DK + 64), "overlap"),
    (dict(dg=DB), "overlap"), (dict(dv=DF), "overlaps an input"), (dict(ws=DQ), "overlap"),
    (dict(ws=MK), "overlaps an input"), (dict(di=DV), "overlap"),
])
def test_backward_refusals(lib, kw, text):
    assert bwd(lib, **kw) == 1 and text in err(lib), err(lib)


def upd(lib, **kw):
    s = sizes()
    a = inputs() | dict(st=ST, slots=8, ss=ONE, idx=IDX, out=OUT, ot=16, oh=8, batch=4) | {
        n: v for n, v in s.items() if n != "T"}
    assert set(kw) <= set(a)
    return lib.gated_delta_rule_update(*(a | kw).values(), None)


@pytest.mark.parametrize("kw,text", [c for c in SHARED if "T" not in c[0]] + [
    (dict(st=None), "NULL"), (dict(out=None), "NULL"), (dict(ss=1), "slots overlap"),
    (dict(idx=None, slots=3), "slots"), (dict(ot=8), "share memory"), (dict(out=V + 4), "overlaps an input"),
    (dict(out=Q), "overlaps an input"), (dict(st=OUT), "overlap"), (dict(st=K), "overlap"),
])
def test_update_refusals(lib, kw, text):
    assert upd(lib, **kw) == 1 and text in err(lib), err(lib)


def test_queries(lib):
    n, m = ctypes.c_int64(), ctypes.c_int64()
    f = lib.gated_delta_rule_checkpoint_rows
    for T, b, dt, want in ((0, 0, 1, 0), (0, 3, 1, 3), (1, 1, 1, 2), (64, 1, 1, 2), (65, 2, 1, 4), (64, 1, 0, 3)):
        assert f(T, b, dt, ctypes.byref(n)) == 0 and n.value == want
    assert f(-1, 1, 0, ctypes.byref(n)) == 1 and f(1, -1, 0, ctypes.byref(n)) == 1
    assert f(1, 1, 2, ctypes.byref(n)) == 1 and f(1, 1, 0, None) == 1
    w = lib.gated_delta_rule_workspace
    assert w(1000, 3, 4, 128, 100, 1, ctypes.byref(n), ctypes.byref(m)) == 0 and 0 < n.value < m.value
    assert n.value % 4 == 0 and m.value > 19 * 4 * 128 * 100
    for bad in ((-1, 1, 1, 1, 1, 0), (1, -1, 1, 1, 1, 0), (1, 1, -1, 1, 1, 0), (1, 1, 1, -1, 1, 0),
                (1, 1, 1, 1, -1, 0), (1, 1, 1, 1, 1, 7)):
        assert w(*bad, ctypes.byref(n), ctypes.byref(m)) == 1
    assert w(1, 1, 1, 1, 1, 0, None, ctypes.byref(m)) == 1 and w(1, 1, 1, 1, 1, 0, ctypes.byref(n), None) == 1


# ---------------------------------------------------------------- layer norm

def lfwd(lib, **kw):
    a = dict(x=Q, xs=16, r=K, rs=16, w=G, b=B, eps=1e-5, ro=DK, ros=16, out=OUT, os=16, rows=4, dim=16, dt=0)
    return lib.layer_norm_fwd(*(a | kw).values(), None)


@pytest.mark.parametrize("kw,text", [
    (dict(rows=-1), ">= 0"), (dict(dim=-1), ">= 0"), (dict(dt=2), "dtype"), (dict(eps=-1.0), "eps"),
    (dict(eps=float("nan")), "eps"), (dict(eps=float("inf")), "eps"), (dict(x=None), "NULL"), (dict(w=None), "NULL"),
    (dict(out=None), "NULL"), (dict(r=None), "without residual"), (dict(xs=-1), "strides"),
    (dict(os=15), "overlap each other"), (dict(ros=0), "overlap each other"), (dict(out=Q + 4), "partially"),
    (dict(ro=K, ros=17), "partially"), (dict(out=G), "weight or bias"), (dict(ro=B + 4), "weight or bias"),
    (dict(ro=OUT), "two outputs"),
])
def test_layer_norm_refusals(lib, kw, text):
    assert lfwd(lib, **kw) == 1 and text in err(lib), err(lib)


def lbwd(lib, **kw):
    a = dict(do=DO, dos=16, x=Q, xs=16, w=G, eps=1e-5, dr=K, drs=16, dx=DQ, dxs=16, dw=DG, db=DB, ws=WS, wsn=64,
             rows=4, dim=16, dt=0)
    return lib.layer_norm_bwd(*(a | kw).values(), None)


@pytest.mark.parametrize("kw,text", [
    (dict(rows=-1), ">= 0"), (dict(dt=5), "dtype"), (dict(eps=-1.0), "eps"), (dict(do=None), "NULL"),
    (dict(dw=None), "NULL"), (dict(ws=None), "NULL"), (dict(dx=None), "NULL"), (dict(wsn=31), "workspace holds"),
    (dict(dos=-1), "strides"), (dict(dxs=8), "overlap each other"), (dict(dx=Q + 4), "partially"),
    (dict(dw=Q), "another buffer"), (dict(db=DG), "another buffer"), (dict(ws=DB), "another buffer"),
    (dict(dx=G), "another buffer"), (dict(ws=DQ), "another buffer"),
])
def test_layer_norm_gradient_refusals(lib, kw, text):
    assert lbwd(lib, **kw) == 1 and text in err(lib), err(lib)


def test_layer_norm_no_ops(lib):
    n = ctypes.c_int64()
    assert lfwd(lib, rows=0) == 0 and lfwd(lib, dim=0) == 0 and lbwd(lib, dim=0) == 0
    assert lfwd(lib, rows=1 << 40, xs=0, rs=0, r=None, ro=None) == 2 and lbwd(lib, dim=(1 << 28) + 1) == 2
    assert lib.layer_norm_bwd_workspace(4, 16, ctypes.byref(n)) == 0 and n.value == 32
    assert lib.layer_norm_bwd_workspace(-1, 16, ctypes.byref(n)) == 1
    assert lib.layer_norm_bwd_workspace(4, 16, None) == 1


# ---------------------------------------------------------------- paged metadata

def meta(lib, **kw):
    a = dict(q=Q, c=K, n=4, free=V, nf=16, bt=ST, bts=8, mb=8, bs=16, qsl=QSL, pad=64, si=DQ, qs=DK, pos=DV, slot=DG,
             used=DB)
    return lib.sconv_paged_metadata(*(a | kw).values(), None)


@pytest.mark.parametrize("kw,text", [
    (dict(n=-1), "negative"), (dict(nf=-1), "negative"), (dict(mb=-1), "negative"), (dict(pad=-1), "negative"),
    (dict(bs=0), "block_size"), (dict(bts=7), "rows of block_table"), (dict(q=None), "NULL"), (dict(c=None), "NULL"),
    (dict(free=None), "NULL"), (dict(bt=None), "NULL"), (dict(qsl=None), "NULL"), (dict(pos=None), "NULL"),
    (dict(slot=None), "NULL"), (dict(bt=Q), "overlaps"), (dict(qsl=ST + 4), "overlaps"), (dict(pos=DG + 8), "overlaps"),
    (dict(si=DK), "overlaps"), (dict(used=K), "overlaps"), (dict(slot=V), "overlaps"),
])
def test_metadata_refusals(lib, kw, text):
    assert meta(lib, **kw) == 1 and text in err(lib), err(lib)


def test_metadata_limits(lib):
    # the buffers of so many rows would overlap: only the launch is too large
    far = {n: (1 << 44) * k for k, n in enumerate(("si", "qs", "pos", "slot"), 2)}
    assert meta(lib, pad=1 << 33, **far) == 2


def test_binding_refuses_host_tensors_and_types():
    q, v, g = torch.zeros(4, 1, 8), torch.zeros(4, 2, 8), torch.zeros(4, 2)
    qsl = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        sc.gated_delta_rule_varlen_fwd(q, q, v, g, g, None, qsl)
    with pytest.raises(ValueError, match="GPU"):
        sc.gated_delta_rule_update(q, q, v, g, g, torch.zeros(4, 2, 8, 8))
    with pytest.raises(ValueError, match="GPU"):
        sc.layer_norm_fwd(torch.zeros(2, 8), torch.ones(8))
    with pytest.raises(ValueError, match="GPU"):
        sc.sconv_paged_metadata(qsl, qsl, qsl, qsl.view(1, 2), 16, qsl, None, None, qsl, qsl)
    with pytest.raises(TypeError, match="element type"):
        sc.gated_delta_rule_checkpoints(q.half(), v.half(), qsl)
