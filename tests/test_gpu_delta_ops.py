"""The gated delta rule on the GPU against the 64-bit reference: prefill,
gradients, one-token update, and a layer that runs them with the conv."""
from __future__ import annotations

import pytest
import torch

import depthwise_causal_conv1d_amd as lib
from tests import delta_ref as D
from tests import layer_ref as R

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
NAN = float("nan")
SENTINEL = -777.0
NAMES = ("dq", "dk", "dv", "dg", "dbeta")


def rand(seed, *shape, dtype=torch.float32, scale=1.0):
    t = torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale
    return t.to(dtype)


def place(t, layout):
    """t [T, heads, channels] on the GPU: dense, as columns of a wider matrix
    from an odd element on, or head after head; NaN around it."""
    T, H, W = t.shape
    n = T * H * W + 64
    if layout == "dense":
        v = torch.full((n,), NAN, dtype=t.dtype, device="cuda")[:n - 64].view(T, H, W)
    elif layout == "columns":
        row = H * W + 13
        v = torch.full((max(T, 1) * row + 3,), NAN, dtype=t.dtype, device="cuda")[3:].as_strided(
            (T, H, W), (row, W, 1), 3)
    else:
        v = torch.full((n,), NAN, dtype=t.dtype, device="cuda")[:n - 64].view(H, T, W).transpose(0, 1)
    return v.copy_(t)


class Case:
    """One packed problem: sequences inside [lead, T), some with an initial
    state, some skipped; NaN wherever nothing may be read."""

    def __init__(self, lens, kh, vh, K, V, dtype, gates="f32", seed=0, inits=(), pads=(), lead=0,
                 trail=0, rate=0.3, scale=None):
        n, dt = len(lens), DT[dtype]
        self.lens, self.kh, self.vh, self.K, self.V = lens, kh, vh, K, V
        self.split, self.scale = dtype == "bf16", scale if scale is not None else K ** -0.5
        self.bounds = [b + lead for b in R.offsets(lens)]
        self.T = T = self.bounds[-1] + trail
        unit = lambda s: torch.nn.functional.normalize(rand(s, T, kh, K), dim=2).to(dt)  # noqa: E731
        self.q, self.k = unit(seed + 1), unit(seed + 2)
        self.v, self.dout = rand(seed + 3, T, vh, V, dtype=dt), rand(seed + 4, T, vh, V, dtype=dt)
        self.g = (-rand(seed + 5, T, vh).abs() * rate).to(DT[gates])
        self.beta = torch.sigmoid(rand(seed + 6, T, vh)).to(DT[gates])
        gen = torch.Generator().manual_seed(seed + 7)
        self.slots = torch.randperm(n + 2, generator=gen)[:n].to(torch.int32)
        self.has = torch.zeros(n, dtype=torch.bool)
        self.has[list(inits)] = True
        self.live = [b not in pads for b in range(n)]
        self.h0, self.dfinal = rand(seed + 8, n, vh, K, V, scale=0.3), rand(seed + 9, n, vh, K, V, scale=0.3)
        self.pool = torch.full((n + 2, vh, K, V), NAN)
        self.inside = torch.zeros(T, dtype=torch.bool)
        for b in range(n):
            if self.live[b]:
                self.inside[self.bounds[b]:self.bounds[b + 1]] = True
                if self.has[b]:
                    self.pool[int(self.slots[b])] = self.h0[b]
            else:
                self.slots[b] = -1
        for t in (self.q, self.k, self.v, self.dout, self.g, self.beta):
            t[~self.inside] = NAN

    def ref(self, grads=True, dfinal=True):
        """Per live sequence: (b, values, bounds)."""
        group = self.vh // self.kh
        for b in range(len(self.lens)):
            if not self.live[b]:
                continue
            c = slice(self.bounds[b], self.bounds[b + 1])
            wide = lambda t: R.f64(t[c]).repeat_interleave(group, 1)  # noqa: E731
            args = wide(self.q), wide(self.k), R.f64(self.v[c]), R.f64(self.g[c]), R.f64(self.beta[c])
            s0 = R.f64(self.h0[b]) * float(self.has[b])
            out, states = D.forward(*args, self.scale, s0)
            if not grads:
                e = D.bounds(*args, self.scale, states, self.split)
                yield b, c, dict(out=out, last=states[-1]), e
                continue
            dout, ds = R.f64(self.dout[c]), R.f64(self.dfinal[b]) * float(dfinal)
            gr = D.backward(dout, *args, self.scale, states, ds)
            e = D.bounds(*args, self.scale, states, self.split, gr, dout, ds)
            gr["dinitial"] = gr["dinitial"] * float(self.has[b])
            for n in ("dq", "dk"):  # summed over the value heads of a key head
                gr[n] = gr[n].unflatten(1, (self.kh, group)).sum(2)
                e[n] = e[n].unflatten(1, (self.kh, group)).sum(2)[..., None].expand_as(gr[n])
                e[n] = e[n] + group * R.EPS * gr[n].abs()
            yield b, c, dict(out=out, last=states[-1], **gr), e

    def gpu(self, layout="dense"):
        d = {n: place(getattr(self, n), layout) for n in ("q", "k", "v", "dout")}
        for n in ("g", "beta"):
            d[n] = place(getattr(self, n)[..., None], layout)[..., 0]
        d |= dict(pool=self.pool.cuda(), slots=self.slots.cuda(), has=self.has.cuda(),
                  qsl=torch.tensor(self.bounds, dtype=torch.int32, device="cuda"))
        return d

    def forward(self, d, layout="dense", out=None, marks=True, states=True):
        out = place(torch.full_like(self.v, SENTINEL), layout) if out is None else out
        m = None
        if marks:
            m = lib.gated_delta_rule_checkpoints(d["k"], d["v"], d["qsl"]).fill_(NAN)
        lib.gated_delta_rule_varlen_fwd(
            d["q"], d["k"], d["v"], d["g"], d["beta"], d["pool"] if states else None, d["qsl"],
            d["slots"], d["has"] if states else None, scale=self.scale, out=out, checkpoints=m)
        return out, m

    def backward(self, d, m, layout="dense", states=True):
        new = {n: place(torch.full_like(getattr(self, n[1:]), SENTINEL), layout)
               for n in ("dq", "dk", "dv")}
        df = di = None
        if states:
            df = torch.full_like(self.pool, NAN)
            for b in range(len(self.lens)):
                if self.live[b]:
                    df[int(self.slots[b])] = self.dfinal[b]
            df, di = df.cuda(), torch.full_like(self.pool, SENTINEL).cuda()
        got = lib.gated_delta_rule_varlen_bwd(
            d["dout"], d["q"], d["k"], d["v"], d["g"], d["beta"], m, d["qsl"], d["slots"],
            d["has"] if states else None, scale=self.scale, dfinal_states=df, dinitial_states=di, **new)
        return dict(zip(NAMES, got)), di

    def check(self, out, pool=None, got=None, di=None, what="", dfinal=True):
        o = out.cpu()
        assert bool((o[~self.inside] == SENTINEL).all()), what + ": wrote outside the sequences"
        host = {n: t.cpu() for n, t in (got or {}).items()}
        for n in ("dq", "dk", "dv"):
            if got:
                assert bool((host[n][~self.inside] == SENTINEL).all()), f"{what} {n}: wrote outside"
        whole = {n: ([], []) for n in ("dg", "dbeta")}
        p = want = w2 = None
        if pool is not None:
            p, want = pool.cpu(), self.pool.clone()
        if di is not None:
            di = di.cpu()
            w2 = torch.full_like(di, SENTINEL)
        for b, c, v, e in self.ref(got is not None, dfinal):
            R.check(o[c], v["out"], e["out"], f"{what} out {b}")
            s = int(self.slots[b])
            if p is not None:
                R.check(p[s], v["last"], e["last"][:, None].expand_as(v["last"]), f"{what} state {b}")
                want[s] = p[s]
            for n in host:
                R.check(host[n][c], v[n], e[n], f"{what} {n} {b}")
                if n in whole:
                    whole[n][0].append(host[n][c]), whole[n][1].append(v[n])
            if di is not None:
                R.check(di[s], v["dinitial"], e["dinitial"][:, None].expand_as(v["dinitial"]),
                        f"{what} dinitial {b}")
                w2[s] = di[s]
        for n, (x, y) in whole.items():
            if x and host and sum(t.numel() for t in y) > 16:
                x, y = torch.cat(x), torch.cat(y)
                lim = D.norm_limit(self.split) + R.half_step(x.dtype)
                assert D.off(x, y) < lim, (what, n, D.off(x, y), lim)
        if p is not None:
            assert torch.equal(R.bits(p), R.bits(want)), what + ": wrote another slot"
        if di is not None:
            assert torch.equal(R.bits(di), R.bits(w2)), what + ": wrote another dinitial"


# lengths around the chunk (64, fp32 32) and its tiles; empty ones between
LENGTHS = [
    dict(lens=[1], inits=(0,)),
    dict(lens=[64, 0, 32, 65, 33], inits=(1, 3), lead=5, trail=7),
    dict(lens=[130, 3, 16, 17], pads=(1,), inits=(0, 2)),
    dict(lens=[0, 0, 200], inits=(0,), trail=1),
]
# key heads, value heads, K, V
SHAPES = [(1, 1, 128, 128), (2, 4, 64, 64), (1, 3, 77, 129), (2, 2, 1, 1), (1, 2, 128, 200), (3, 3, 40, 16),
          (1, 1, 16, 300)]


@pytest.mark.parametrize("dtype,gates", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_prefill_and_gradients(shape, dtype, gates):
    for n, spec in enumerate(LENGTHS):
        c = Case(**spec, **dict(zip(("kh", "vh", "K", "V"), SHAPES[shape])), dtype=dtype, gates=gates,
                 seed=10 * n + shape)
        layout = ("dense", "columns", "heads")[(n + shape) % 3]
        d = c.gpu(layout)
        out, m = c.forward(d, layout)
        got, di = c.backward(d, m, layout)
        c.check(out, d["pool"], got, di, f"{spec['lens']} {layout}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["dense", "columns", "heads"])
def test_without_states_and_in_place(layout, dtype):
    c = Case([70, 0, 129], 2, 4, 64, 48, dtype, seed=3, lead=2)
    d = c.gpu(layout)
    out, m = c.forward(d, layout, states=False)
    got, di = c.backward(d, m, layout, states=False)
    c.check(out, None, got, None, layout, dfinal=False)
    v = d["v"].clone()
    assert c.forward(d, layout, out=d["v"], marks=False, states=False)[0] is d["v"]
    assert torch.equal(R.bits(d["v"][c.inside.cuda()]), R.bits(out[c.inside.cuda()]))
    d["v"] = v


def test_long_sequences_among_many():
    """Many chunks, many sequences, a workgroup of columns that ends early."""
    c = Case([700, 1, 0, 64, 311, 2, 128], 2, 4, 128, 72, "bf16", seed=5, inits=(0, 4, 6), rate=0.02)
    d = c.gpu()
    out, m = c.forward(d)
    got, di = c.backward(d, m)
    c.check(out, d["pool"], got, di, "many")
    # equal inputs give equal bits
    d2 = c.gpu()
    out2, m2 = c.forward(d2)
    got2, di2 = c.backward(d2, m2)
    for a, b in [(out, out2), (d["pool"], d2["pool"]), (di, di2)] + [(got[n], got2[n]) for n in NAMES]:
        a, b = torch.nan_to_num(a, 7.0), torch.nan_to_num(b, 7.0)
        inside = c.inside.cuda()
        if a.shape[0] == c.T:
            a, b = a[inside], b[inside]
        assert torch.equal(R.bits(a), R.bits(b))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kh,vh,lens", [(1, 40, [70, 5]), (3, 9, [65, 0, 33])])
def test_heads_that_share_a_key_head(kh, vh, lens, dtype):
    """More workgroups of one sequence and key head than an XCD has CUs, and
    sequences and key heads that the XCDs do not divide evenly."""
    c = Case(lens, kh, vh, 24, 72 if kh > 1 else 20, dtype, seed=21, inits=(0,))
    d = c.gpu()
    out, m = c.forward(d)
    got, di = c.backward(d, m)
    c.check(out, d["pool"], got, di, "shared")


@pytest.mark.parametrize("lead", [0, 5])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_inputs_and_gradients_as_columns_of_one_matrix(dtype, lead):
    """q, k, v as columns of a conv's output and their gradients as columns of
    another matrix (aligned rows, and rows from an odd element on); gates and
    betas as columns too."""
    c = Case([70, 3, 64], 2, 4, 32, 48, dtype, gates=dtype, seed=12, inits=(1,))
    wide = [2 * 32, 2 * 32, 4 * 48]

    def columns(*ts):
        T, n = ts[0].shape[0], sum(t[0].numel() for t in ts)
        row = n + lead
        m = torch.full((T * row + lead,), NAN, dtype=ts[0].dtype, device="cuda")[lead:].as_strided(
            (T, n), (row, 1), lead)
        return [p.view(t.shape).copy_(t) for p, t in zip(m.split([t[0].numel() for t in ts], 1), ts)]

    assert wide == [t[0].numel() for t in (c.q, c.k, c.v)]
    d = c.gpu()
    d["q"], d["k"], d["v"] = columns(c.q, c.k, c.v)
    d["g"], d["beta"] = (t[..., 0] for t in columns(c.g[..., None], c.beta[..., None]))
    out = place(torch.full_like(c.v, SENTINEL), "dense")
    m = lib.gated_delta_rule_checkpoints(d["k"], d["v"], d["qsl"])
    args = d["q"], d["k"], d["v"], d["g"], d["beta"]
    lib.gated_delta_rule_varlen_fwd(*args, d["pool"], d["qsl"], d["slots"], d["has"], scale=c.scale,
                                    out=out, checkpoints=m)
    new = columns(*(torch.full_like(t, SENTINEL) for t in (c.q, c.k, c.v)))
    got = dict(zip(NAMES, lib.gated_delta_rule_varlen_bwd(
        d["dout"], *args, m, d["qsl"], d["slots"], d["has"], scale=c.scale,
        dq=new[0], dk=new[1], dv=new[2])))
    c.check(out, d["pool"], got, None, "columns", dfinal=False)


@pytest.mark.parametrize("heads,batch", [(40, 9), (3, 2)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_workgroups_of_both_widths(dtype, heads, batch):
    """Enough heads and sequences for eight computing waves a workgroup, and too
    few; more columns than one workgroup takes; equal bits in both where the
    sequence is the same."""
    lens = [40, 65] + [1] * (batch - 2)
    c = Case(lens, 1, heads, 32, 136, dtype, seed=13, inits=(1,))
    d = c.gpu()
    out, m = c.forward(d)
    got, di = c.backward(d, m)
    o, state = out.clone(), d["pool"].clone()
    # the first two sequences and three heads alone
    few = {n: d[n][:105, :3] for n in ("v", "g", "beta")}
    st = torch.full((2, 3, 32, 136), NAN, device="cuda")
    st[1] = c.h0[1, :3].cuda()
    alone = lib.gated_delta_rule_varlen_fwd(d["q"][:105], d["k"][:105], few["v"], few["g"], few["beta"], st,
                                            d["qsl"][:3].clone(), None, d["has"][:2].clone(), scale=c.scale)
    assert torch.equal(R.bits(alone), R.bits(o[:105, :3]))
    for b in (0, 1):
        assert torch.equal(R.bits(st[b]), R.bits(state[int(c.slots[b]), :3]))
    if heads == 3:
        c.check(out, d["pool"], got, di, "narrow")
    else:  # a few heads of the gradients: the reference of all takes minutes
        few = Case.__new__(Case)
        few.__dict__.update(c.__dict__)
        few.vh = 2
        few.v, few.dout, few.g, few.beta = (t[:, :2] for t in (c.v, c.dout, c.g, c.beta))
        few.h0, few.dfinal, few.pool = (t[:, :2] for t in (c.h0, c.dfinal, c.pool))
        part = {n: got[n][:, :2] for n in ("dv", "dg", "dbeta")}
        for b, s, v, e in few.ref():
            R.check(out[s, :2], v["out"], e["out"], f"wide out {b}")
            for n, t in part.items():
                R.check(t[s], v[n], e[n], f"wide {n} {b}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_closed_open_and_strong_gates(dtype):
    """g of 0, -inf and far below -200, beta of 0, 1 and 2: closed gates forget
    everything before them, and their dg is zero."""
    c = Case([150], 1, 2, 64, 32, dtype, seed=6, inits=(0,))
    c.g[:] = 0.0
    c.g[40] = -float("inf")
    c.g[41] = -1e30
    c.g[100] = -150.0
    c.beta[10:20], c.beta[20:30], c.beta[30:35] = 0.0, 1.0, 2.0
    d = c.gpu()
    out, m = c.forward(d)
    got, di = c.backward(d, m)
    c.g[c.g < -200] = -200.0  # e^-200 is zero in fp32 and what the reference sees
    c.check(out, d["pool"], got, di, "gates")
    assert bool((got["dg"][40:42] == 0).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_nan_stays_in_its_sequence_and_column(dtype):
    c = Case([90, 90, 90], 1, 2, 64, 64, dtype, seed=7)
    clean, _ = c.forward(c.gpu(), marks=False, states=False)
    d = c.gpu()
    d["v"][100, 1, 5] = NAN
    out, _ = c.forward(d, marks=False, states=False)
    bad = out.isnan()
    assert bool(bad[100:180, 1, 5].all())
    bad[64 + 26:180, 1, 5] = False  # its column of the chunk it lies in, and on
    assert not bool(bad.any())
    keep = ~out.isnan()
    assert torch.equal(R.bits(out[keep]), R.bits(clean[keep]))
    d = c.gpu()
    d["k"][100, 0, 3] = NAN
    out, _ = c.forward(d, marks=False, states=False)
    assert torch.equal(R.bits(out[:90]), R.bits(clean[:90]))
    assert torch.equal(R.bits(out[180:]), R.bits(clean[180:]))
    assert bool(out[100:180].isnan().all())


@pytest.mark.parametrize("dtype,gates", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("rows,shape", [(1, (1, 1, 1, 1)), (3, (2, 4, 64, 64)), (9, (1, 3, 77, 129)),
                                        (5, (2, 2, 128, 128)), (4, (1, 2, 100, 260)), (70, (1, 1, 16, 4))])
def test_update(rows, shape, dtype, gates):
    pads = (1,) if rows > 2 else ()
    for layout in ("dense", "columns", "heads"):
        c = Case([1] * rows, *shape, dtype, gates, seed=rows, inits=range(rows), pads=pads)
        d = c.gpu(layout)
        out = place(torch.full_like(c.v, SENTINEL), layout)
        lib.gated_delta_rule_update(d["q"], d["k"], d["v"], d["g"], d["beta"], d["pool"], d["slots"],
                                    scale=c.scale, out=out)
        c.check(out, d["pool"], what=layout)


def test_update_pools_at_any_slot_stride():
    for extra in (4, 1):
        c = Case([1] * 4, 1, 2, 32, 32, "f32", seed=2, inits=range(4))
        d = c.gpu()
        one = 2 * 32 * 32
        pool = torch.full((6 * (one + extra),), NAN, device="cuda").as_strided(
            (6, 2, 32, 32), (one + extra, 1024, 32, 1))
        pool.copy_(d["pool"])
        out = place(torch.full_like(c.v, SENTINEL), "dense")
        lib.gated_delta_rule_update(d["q"], d["k"], d["v"], d["g"], d["beta"], pool, d["slots"],
                                    scale=c.scale, out=out)
        c.check(out, pool, what=str(extra))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decode_continues_a_prefill(dtype):
    """A prompt of 70 tokens and 5 decoded ones against 75 at once."""
    c = Case([75], 1, 2, 64, 64, dtype, seed=8)
    d = c.gpu()
    cut = torch.tensor([0, 70], dtype=torch.int32, device="cuda")
    slots = d["slots"]
    out = place(torch.full_like(c.v, SENTINEL), "dense")
    lib.gated_delta_rule_varlen_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], d["pool"], cut, slots,
                                    scale=c.scale, out=out)
    for t in range(70, 75):
        s = slice(t, t + 1)
        lib.gated_delta_rule_update(d["q"][s], d["k"][s], d["v"][s], d["g"][s], d["beta"][s],
                                    d["pool"], slots, scale=c.scale, out=out[s])
    c.check(out, d["pool"], what="decode")


def test_empty_calls():
    e = dict(device="cuda")
    q, v, g = torch.empty(0, 1, 8, **e), torch.empty(0, 2, 4, **e), torch.empty(0, 2, **e)
    q0 = torch.zeros(1, dtype=torch.int32, **e)
    assert lib.gated_delta_rule_varlen_fwd(q, q, v, g, g, None, q0).shape == (0, 2, 4)
    q2 = torch.zeros(3, dtype=torch.int32, **e)
    st = torch.ones(2, 2, 8, 4, **e)
    has = torch.tensor([True, False], **e)
    m = lib.gated_delta_rule_checkpoints(q, v, q2)
    lib.gated_delta_rule_varlen_fwd(q, q, v, g, g, st, q2, None, has, checkpoints=m)
    assert bool((st[0] == 1).all()) and bool((st[1] == 0).all())
    di = torch.full_like(st, 5.0)
    lib.gated_delta_rule_varlen_bwd(v, q, q, v, g, g, m, q2, None, has,
                                    dfinal_states=torch.full_like(st, 3.0), dinitial_states=di)
    assert bool((di[0] == 3).all()) and bool((di[1] == 0).all())
    assert lib.gated_delta_rule_update(q, q, v, g, g, st).shape == (0, 2, 4)


# ---------------------------------------------------------------- a layer, graphs, streams

KH, VH, HK, HV = 1, 2, 16, 16
WIDTH = 2 * KH * HK + VH * HV


def split_heads(u):
    """q, k, v as columns of the conv's output rows [T, WIDTH]."""
    T = u.shape[0]
    q, k, v = u.split([KH * HK, KH * HK, VH * HV], 1)
    return q.view(T, KH, HK), k.view(T, KH, HK), v.view(T, VH, HV)


def layer_step(t):
    """layer norm -> conv -> unit q and k -> delta rule, and back."""
    y = lib.layer_norm_fwd(t["x"], t["nw"], t["nb"], 1e-5, residual=t["res"], residual_out=t["sum"])
    u = y.clone()
    lib.causal_conv1d_varlen_fwd(u.t(), t["cw"], t["cb"], t["cstate"], t["qsl"], None, None, True)
    q, k, v = split_heads(u)
    T = u.shape[0]
    unit = t["unit"]
    qn = lib.rms_norm_fwd(q.reshape(-1, HK), unit, 1e-6).view(T, KH, HK)
    kn = lib.rms_norm_fwd(k.reshape(-1, HK), unit, 1e-6).view(T, KH, HK)
    marks = lib.gated_delta_rule_checkpoints(kn, v, t["qsl"])
    out = lib.gated_delta_rule_varlen_fwd(qn, kn, v, t["g"], t["beta"], None, t["qsl"], checkpoints=marks)
    du = torch.empty_like(u)
    dq, dk, dv = split_heads(du)
    dqn, dkn, _, dg, dbeta = lib.gated_delta_rule_varlen_bwd(
        t["dout"], qn, kn, v, t["g"], t["beta"], marks, t["qsl"], dv=dv)
    for d, x, to in ((dqn, q, dq), (dkn, k, dk)):
        to.copy_(lib.rms_norm_bwd(d.view(-1, HK), x.reshape(-1, HK), unit, 1e-6)[0].view(T, KH, HK))
    dc, dw, db = lib.causal_conv1d_varlen_bwd(du.t(), y.t(), t["cw"], t["cb"], None, t["qsl"], None,
                                              None, True)
    dx, dnw, dnb = lib.layer_norm_bwd(dc.t(), t["sum"], t["nw"], 1e-5)
    return dict(out=out, dg=dg, dbeta=dbeta, dw=dw, db=db, dx=dx, dnw=dnw, dnb=dnb)


def layer_inputs(seed, lens=(130, 0, 100, 1)):
    b = R.offsets(lens)
    T = b[-1]
    t = dict(x=rand(seed, T, WIDTH), res=rand(seed + 1, T, WIDTH), nw=rand(seed + 2, WIDTH) * 0.1 + 1,
             nb=rand(seed + 3, WIDTH, scale=0.1), cw=rand(seed + 4, WIDTH, 4, scale=0.5),
             cb=rand(seed + 5, WIDTH, scale=0.1), g=-rand(seed + 6, T, VH).abs() * 0.3,
             beta=torch.sigmoid(rand(seed + 7, T, VH)), dout=rand(seed + 8, T, VH, HV))
    d = {k: v.cuda() for k, v in t.items()}
    d["unit"] = torch.full((HK,), HK ** -0.5, device="cuda")
    d["sum"] = torch.empty_like(d["x"])
    d["cstate"] = torch.zeros(len(lens), WIDTH, 3, device="cuda")
    d["qsl"] = torch.tensor(b, dtype=torch.int32, device="cuda")
    return t, d, b


def test_layer_runs_together():
    t, d, b = layer_inputs(40)
    got = layer_step(d)
    w = {k: v.double().requires_grad_() for k, v in t.items() if k != "dout"}
    s = w["x"] + w["res"]
    y = torch.nn.functional.layer_norm(s, (WIDTH,), w["nw"], w["nb"], 1e-5)
    outs = []
    for lo, hi in zip(b[:-1], b[1:]):
        if hi == lo:
            continue
        u = torch.cat([torch.zeros(3, WIDTH, dtype=torch.float64), y[lo:hi]])
        z = w["cb"] + sum(w["cw"][:, j] * u[j:j + hi - lo] for j in range(4))
        q, k, v = split_heads(z * torch.sigmoid(z))
        q, k = (x / torch.sqrt((x * x).mean(2, keepdim=True) + 1e-6) * HK ** -0.5 for x in (q, k))
        q, k = (x.repeat_interleave(VH // KH, 1) for x in (q, k))
        outs.append(D.forward(q, k, v, w["g"][lo:hi], w["beta"][lo:hi], HK ** -0.5,
                              torch.zeros(VH, HK, HV, dtype=torch.float64))[0])
    out = torch.cat(outs)
    (out * t["dout"].double()).sum().backward()
    # four operators in a row in 32 bits: norms as norm_limit() counts them, 8 of them
    for name, ref in (("out", out), ("dg", w["g"].grad), ("dbeta", w["beta"].grad),
                      ("dw", w["cw"].grad), ("db", w["cb"].grad), ("dx", w["x"].grad),
                      ("dnw", w["nw"].grad), ("dnb", w["nb"].grad)):
        assert D.off(got[name].cpu(), ref.detach()) < 8 * D.norm_limit(False), name


def test_layer_in_a_graph_and_on_another_stream():
    """Captured once, replayed on new inputs with eager work between: equal
    bits each time; the same on a side stream."""
    _, d, _ = layer_inputs(60)
    lib.sconv_init()
    warm = torch.cuda.Stream()
    with torch.cuda.stream(warm):
        layer_step(d)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    d["cstate"].zero_()
    with torch.cuda.graph(graph):
        held = layer_step(d)
    for seed in (70, 80, 90):
        _, new, _ = layer_inputs(seed)
        for k in d:
            if k not in ("qsl", "sum"):
                d[k].copy_(new[k])
        graph.replay()
        torch.cuda.synchronize()
        replayed = {k: v.clone() for k, v in held.items()}
        eager = layer_step(new)
        with torch.cuda.stream(warm):
            warm.wait_stream(torch.cuda.current_stream())
            new["cstate"].zero_()
            side = layer_step(new)
        torch.cuda.synchronize()
        for k in held:
            assert torch.equal(R.bits(replayed[k]), R.bits(eager[k])), (seed, k)
            assert torch.equal(R.bits(side[k]), R.bits(eager[k])), (seed, k, "side stream")


def test_two_streams_and_two_graphs_at_once():
    """Calls in flight on two streams, and two captured graphs replayed in turn
    and side by side, keep their own workspaces."""
    ins = [layer_inputs(s, lens=(300, 200))[1] for s in (100, 110)]
    want = []
    for d in ins:
        want.append({k: v.clone() for k, v in layer_step(d).items()})
        d["cstate"].zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None, None]
    for _ in range(5):
        for k in (0, 1):
            with torch.cuda.stream(streams[k]):
                got[k] = layer_step(ins[k])
    torch.cuda.synchronize()
    for k in (0, 1):
        for n in want[k]:
            assert torch.equal(R.bits(got[k][n]), R.bits(want[k][n])), (k, n, "streams")
    graphs, held = [], []
    for k in (0, 1):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held.append(layer_step(ins[k]))
        graphs.append(g)
    for turn in range(4):
        for k in (0, 1):
            with torch.cuda.stream(streams[k if turn % 2 else 0]):
                graphs[k].replay()
        torch.cuda.synchronize()
        for k in (0, 1):
            for n in want[k]:
                assert torch.equal(R.bits(held[k][n]), R.bits(want[k][n])), (turn, k, n, "graphs")


def test_strides_and_slots_past_32_bits():
    """Tokens and heads whose element offsets pass 2^31, slots whose byte
    offsets pass 2^32."""
    step = (1 << 31) + 8
    big = torch.empty(2 * step + 65536, dtype=torch.bfloat16, device="cuda")
    for heads in (False, True):
        c = Case([3], 1, 2, 64, 64, "bf16", seed=9) if heads else Case([3], 1, 1, 64, 64, "bf16", seed=9)
        d = c.gpu()

        def far(t, at):
            T, H, W = t.shape
            st = (W, step, 1) if heads and H > 1 else (step, W, 1)
            return big[at:].as_strided(t.shape, st).copy_(t)

        d["q"], d["k"] = (far(d[n], i * 1024) if not heads else d[n] for i, n in enumerate(("q", "k")))
        d["v"], d["dout"] = far(d["v"], 2048), far(d["dout"], 4096)
        out, m = c.forward(d, out=far(torch.full_like(d["v"], SENTINEL), 8192))
        new = dict(dv=far(torch.empty_like(d["v"]), 12288))
        got = dict(zip(NAMES, lib.gated_delta_rule_varlen_bwd(
            d["dout"], d["q"], d["k"], d["v"], d["g"], d["beta"], m, d["qsl"], scale=c.scale, **new)))
        c.check(out, d["pool"], got, None, f"far {heads}", dfinal=False)
    c = Case([1, 1], 1, 1, 16, 16, "f32", seed=4, inits=(0, 1))
    d = c.gpu()
    pool = big.view(torch.float32)[64:].as_strided((2, 1, 16, 16), ((1 << 31) - 4096, 256, 16, 1)).copy_(c.h0)
    out = place(torch.full_like(c.v, SENTINEL), "dense")
    lib.gated_delta_rule_update(d["q"], d["k"], d["v"], d["g"], d["beta"], pool, scale=c.scale, out=out)
    back = torch.full_like(c.pool, NAN)
    for b in (0, 1):
        back[int(c.slots[b])] = pool[b].cpu()
    c.check(out, back, what="far slots")


def test_padded_batch_of_empty_sequences():
    for n in (1, 70):
        lens = [90, 130] + [0] * n
        c = Case(lens, 1, 2, 40, 24, "f32", seed=50, inits=range(0, n + 2, 3), pads=range(n, n + 2), trail=9)
        d = c.gpu()
        out, m = c.forward(d)
        got, di = c.backward(d, m)
        c.check(out, d["pool"], got, di, str(n))
