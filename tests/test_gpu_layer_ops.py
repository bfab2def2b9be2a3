"""The layer operators on the GPU against the 64-bit references: gated linear
recurrence (prefill, gradients, one-token update), the conv's gradients, the
RMS norm, and a layer that runs them together."""
from __future__ import annotations

import pytest
import torch

import depthwise_causal_conv1d_amd as lib
from tests import layer_ref as R

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
NAN = float("nan")
SENTINEL = -777.0
LAYOUTS = ["channel", "channel_odd", "token", "token_odd", "strided"]


def rand(seed, *shape, dtype=torch.float32, scale=1.0):
    t = torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale
    return t.to(dtype)


def place(t, layout, extra=0):
    """t [dim, T] on the GPU in a layout: channel-major with aligned rows, the
    same from an odd offset, rows of tokens with aligned or odd rows, every
    third element of a larger buffer."""
    dim, T = t.shape
    dev = "cuda"
    if layout == "channel":
        buf = torch.full((dim, (T + 15) // 8 * 8), NAN, dtype=t.dtype, device=dev)
        v = buf[:, :T]
    elif layout == "channel_odd":
        v = torch.full((dim * (T + 1) + 1,), NAN, dtype=t.dtype, device=dev)[1:].as_strided(
            (dim, T), (T + 1, 1), 1)
    elif layout == "token":
        buf = torch.full((T, (dim + 15) // 8 * 8), NAN, dtype=t.dtype, device=dev)
        v = buf[:, :dim].t()
    elif layout == "token_odd":
        v = torch.full((T * (dim + 1) + 1,), NAN, dtype=t.dtype, device=dev).as_strided(
            (dim, T), (1, dim + 1), 1)
    else:
        v = torch.full((3 * dim * T + 3,), NAN, dtype=t.dtype, device=dev).as_strided(
            (dim, T), (3, 3 * dim), 1)
    v.copy_(t)
    return v


class Rec:
    """One recurrence problem: sequences inside [lead, total), some with an
    initial state, some skipped; NaN wherever nothing may be read."""

    def __init__(self, lens, dim, dtype, seed=0, inits=(), pads=(), lead=0, trail=0, gate_scale=1.5,
                 scale=8.0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.dim, self.scale = lens, dim, scale
        self.bounds = [v + lead for v in R.offsets(lens)]
        self.T = self.bounds[-1] + trail
        n = len(lens)
        dt = DT[dtype]
        self.x, self.ga, self.gx, self.dout = (
            rand(seed + k + 1, dim, self.T, dtype=dt, scale=s)
            for k, s in ((0, 1.0), (1, gate_scale), (2, gate_scale), (3, 1.0)))
        a = 0.85 + 0.149 * torch.rand(dim, generator=g)
        self.decay = torch.log(torch.expm1(-torch.log(a) / 8.0))
        self.slots = torch.randperm(n + 3, generator=g)[:n].to(torch.int32)
        self.pads = list(pads)
        self.live = [b not in self.pads for b in range(n)]
        self.has = torch.zeros(n, dtype=torch.bool)
        self.has[list(inits)] = True
        for b in self.pads:
            self.slots[b] = -1
            for t in (self.x, self.ga, self.gx, self.dout):
                t[:, self.bounds[b]:self.bounds[b + 1]] = NAN
        for t in (self.x, self.ga, self.gx, self.dout):
            t[:, :lead] = NAN
            t[:, self.bounds[-1]:] = NAN
        self.h0 = rand(seed + 9, n, dim)
        self.dfinal = rand(seed + 10, n, dim)
        self.pool = torch.full((n + 3, dim), NAN)
        for b in range(n):
            if self.live[b] and self.has[b]:
                self.pool[int(self.slots[b])] = self.h0[b]
        self.inside = torch.zeros(self.T, dtype=torch.bool)
        for b in range(n):
            if self.live[b]:
                self.inside[self.bounds[b]:self.bounds[b + 1]] = True
        # the reference sees zeros in skipped places
        z = lambda t: R.f64(torch.where(self.inside, t, torch.zeros_like(t)))  # noqa: E731
        start = R.f64(self.h0) * self.has[:, None]
        self.f = R.recurrence(z(self.x), z(self.ga), z(self.gx), self.decay, scale, self.bounds, start)
        self.z = z

    def gpu(self, layout):
        return dict(x=place(self.x, layout), ga=place(self.ga, layout), gx=place(self.gx, layout),
                    dout=place(self.dout, layout), decay=self.decay.cuda(), pool=self.pool.cuda(),
                    qsl=torch.tensor(self.bounds, dtype=torch.int32, device="cuda"),
                    slots=self.slots.cuda(), has=self.has.cuda())

    def forward(self, d, layout, out=None, marks=True, states=True):
        out = place(torch.full_like(self.x, SENTINEL), layout) if out is None else out
        m = lib.gated_linear_recurrence_checkpoints(d["x"], d["qsl"]) if marks else None
        lib.gated_linear_recurrence_varlen_fwd(
            d["x"], d["ga"], d["gx"], d["decay"], d["pool"] if states else None, d["qsl"],
            d["slots"], d["has"] if states else None, decay_scale=self.scale, out=out,
            checkpoints=m)
        return out, m

    def check_forward(self, out, pool, what=""):
        o = out.cpu()
        R.check(o[:, self.inside], self.f["h"][:, self.inside], self.f["eh"][:, self.inside],
                what + " out")
        outside = o[:, ~self.inside]
        assert bool((outside == SENTINEL).all()), what + ": wrote outside the sequences"
        if pool is None:
            return
        p, want = pool.cpu(), self.pool.clone()
        for b in range(len(self.lens)):
            if self.live[b]:
                s = int(self.slots[b])
                R.check(p[s], self.f["last"][b], self.f["elast"][b], f"{what} state {b}")
                want[s] = p[s]
        assert torch.equal(R.bits(p), R.bits(want)), what + ": wrote another slot"

    def check_backward(self, got, dinitial, what=""):
        ref = R.recurrence_grad(self.f, self.z(self.dout), self.z(self.x), self.decay, self.scale,
                                self.bounds, R.f64(self.dfinal), R.f64(self.has.double()))
        for name in ("dx", "dgate_a", "dgate_x"):
            g, (v, e) = got[name].cpu(), ref[name]
            R.check(g[:, self.inside], v[:, self.inside], e[:, self.inside], f"{what} {name}")
            assert bool((g[:, ~self.inside] == SENTINEL).all()), f"{what} {name}: wrote outside"
        # skipped sequences have no part in the sum (their reference terms are zero: x and dout are)
        v, e = self._ddecay(ref)
        R.check(got["ddecay"], v, e, what + " ddecay")
        di = dinitial.cpu()
        for b in range(len(self.lens)):
            if self.live[b]:
                s = int(self.slots[b])
                R.check(di[s], ref["dinitial"][0][b], ref["dinitial"][1][b], f"{what} dinitial {b}")
                di[s] = SENTINEL
        assert bool((di == SENTINEL).all()), what + ": dinitial wrote another slot"

    def _ddecay(self, ref):
        if not self.pads:
            return ref["ddecay"]
        # a skipped sequence's dfinal must not enter: take it out of the reference
        df = R.f64(self.dfinal).clone()
        df[self.pads] = 0
        again = R.recurrence_grad(self.f, self.z(self.dout), self.z(self.x), self.decay, self.scale,
                                  self.bounds, df, R.f64(self.has.double()))
        return again["ddecay"]

    def backward(self, d, m, layout):
        outs = {n: place(torch.full_like(self.x, SENTINEL), layout)
                for n in ("dx", "dgate_a", "dgate_x")}
        df = torch.full_like(d["pool"], NAN)
        for b in range(len(self.lens)):
            if self.live[b]:
                df[int(self.slots[b])] = self.dfinal[b].cuda()
        di = torch.full_like(d["pool"], SENTINEL)
        _, _, _, dd = lib.gated_linear_recurrence_varlen_bwd(
            d["dout"], d["x"], d["ga"], d["gx"], d["decay"], m, d["qsl"], d["slots"], d["has"],
            decay_scale=self.scale, dfinal_states=df, dinitial_states=di, **outs)
        return dict(outs, ddecay=dd), di


LENGTHS = [
    ([1], (), ()),
    ([0, 1, 2, 0], (0, 2), ()),
    ([127, 128, 129], (1,), ()),
    ([511, 513, 7, 512], (0, 3), (2,)),
    ([3, 0, 1300, 1, 40], (1, 2), (4,)),
]


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("which", range(len(LENGTHS)))
def test_recurrence_prefill_and_gradients(which, dtype, layout):
    lens, inits, pads = LENGTHS[which]
    dim = [1, 3, 66, 40, 129][(which + LAYOUTS.index(layout)) % 5]
    c = Rec(lens, dim, dtype, seed=which, inits=inits, pads=pads, lead=which % 3, trail=which % 2)
    d = c.gpu(layout)
    out, m = c.forward(d, layout)
    c.check_forward(out, d["pool"], layout)
    got, di = c.backward(d, m, layout)
    c.check_backward(got, di, layout)


@pytest.mark.parametrize("layout", ["channel", "token"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_recurrence_long_sequence(dtype, layout):
    """Thousands of tokens of slow decay: many tiles, one sequence."""
    c = Rec([6007], 16, dtype, seed=3, inits=(0,))
    d = c.gpu(layout)
    out, m = c.forward(d, layout)
    c.check_forward(out, d["pool"], layout)
    got, di = c.backward(d, m, layout)
    c.check_backward(got, di, layout)


@pytest.mark.parametrize("dim,batch", [(256, 1), (520, 3), (64, 40), (2048, 1)])
@pytest.mark.parametrize("layout", ["channel", "token"])
def test_recurrence_launch_shapes(layout, dim, batch):
    """Few and many rows of channels, one and many sequences."""
    lens = [(37 * b) % 300 + 1 for b in range(batch)]
    c = Rec(lens, dim, "bf16", seed=batch, inits=range(0, batch, 2))
    d = c.gpu(layout)
    out, m = c.forward(d, layout)
    c.check_forward(out, d["pool"], layout)
    got, di = c.backward(d, m, layout)
    c.check_backward(got, di, layout)


# Few long sequences in rows are cut into segments of 128 rows and more:
# sequences that end at, before and after a cut, several cuts long, inside one
# segment, empty at a cut and at both ends, skipped.
SEGMENTED = [
    ([128, 1280, 0, 128, 1800], (0, 1), ()),
    ([0, 1000, 3, 0, 2000, 127, 1900, 0], (1, 2, 4, 7), (5,)),
    ([2049], (), ()),
    ([700, 0, 900, 1664, 1], (0, 2, 3), (2,)),
]


@pytest.mark.parametrize("layout", ["token", "token_odd", "channel"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("which", range(len(SEGMENTED)))
def test_recurrence_segments(which, dtype, layout):
    lens, inits, pads = SEGMENTED[which]
    c = Rec(lens, [6, 130, 64, 65][which], dtype, seed=20 + which, inits=inits, pads=pads,
            lead=[0, 5, 0, 64][which], trail=which % 2)
    d = c.gpu(layout)
    out, m = c.forward(d, layout)
    c.check_forward(out, d["pool"], layout)
    got, di = c.backward(d, m, layout)
    c.check_backward(got, di, layout)
    # state gradients in place, and the forward in place: the same bits
    df = torch.full_like(d["pool"], NAN)
    for b in range(len(lens)):
        if c.live[b]:
            df[int(c.slots[b])] = c.dfinal[b].cuda()
    again = lib.gated_linear_recurrence_varlen_bwd(
        d["dout"], d["x"], d["ga"], d["gx"], d["decay"], m, d["qsl"], d["slots"], d["has"],
        decay_scale=c.scale, dfinal_states=df, dinitial_states=df)
    live = [int(c.slots[b]) for b in range(len(lens)) if c.live[b]]
    assert torch.equal(R.bits(df[live]), R.bits(di[live]))
    for g, name in zip(again, ("dx", "dgate_a", "dgate_x")):
        assert torch.equal(R.bits(g)[:, c.inside], R.bits(got[name])[:, c.inside])
    assert torch.equal(R.bits(again[3]), R.bits(got["ddecay"]))
    d["pool"] = c.pool.cuda()
    x = d["x"]
    lib.gated_linear_recurrence_varlen_fwd(x, d["ga"], d["gx"], d["decay"], d["pool"], d["qsl"],
                                           d["slots"], d["has"], decay_scale=c.scale, out=x)
    assert torch.equal(R.bits(x)[:, c.inside], R.bits(out)[:, c.inside])


def test_recurrence_segments_equal_whole_sequences():
    """The C entry without a workspace walks each sequence alone: the results of
    both ways, held to one bound by the tests above, agree to a few units."""
    c = Rec([1500, 900], 64, "f32", seed=31, inits=(0,))
    d = c.gpu("token")
    out, _ = c.forward(d, "token", marks=False)
    from depthwise_causal_conv1d_amd import _lib
    alone = torch.empty_like(d["x"])
    pool = c.pool.cuda()
    pl = lambda t: (t.data_ptr(), *t.stride())  # noqa: E731
    rc = _lib.load().gated_linear_recurrence_varlen_fwd(
        *pl(d["x"]), *pl(d["ga"]), *pl(d["gx"]), d["decay"].data_ptr(), 8.0, pool.data_ptr(),
        pool.shape[0], pool.stride(0), d["qsl"].data_ptr(), 2, d["slots"].data_ptr(),
        d["has"].view(torch.uint8).data_ptr(), *pl(alone), None, 0, None, 0, 64, c.T, 0, -1,
        torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    c.check_forward(alone, pool, "alone")
    assert float((alone - out).abs().max()) <= float(2 * c.f["eh"].max())


@pytest.mark.parametrize("layout", LAYOUTS)
def test_recurrence_in_place_and_without_states(layout):
    c = Rec([300, 5, 600], 24, "bf16", seed=5)
    d = c.gpu(layout)
    out, _ = c.forward(d, layout, marks=False, states=False)
    c.check_forward(out, None, layout)
    lib.gated_linear_recurrence_varlen_fwd(d["x"], d["ga"], d["gx"], d["decay"], None, d["qsl"],
                                           out=d["x"])
    assert torch.equal(R.bits(d["x"]), R.bits(out))


@pytest.mark.parametrize("layout", ["channel", "token"])
def test_recurrence_mixed_layouts_and_shared_projection(layout):
    """x in one layout, the gates as two column blocks of one projection, the
    gate gradients as two column blocks of one buffer."""
    c = Rec([200, 129], 32, "bf16", seed=6)
    d = c.gpu(layout)
    proj = torch.empty(c.T, 64, dtype=torch.bfloat16, device="cuda")
    proj[:, :32], proj[:, 32:] = c.ga.t(), c.gx.t()
    d["ga"], d["gx"] = proj[:, :32].t(), proj[:, 32:].t()
    out, m = c.forward(d, layout)
    c.check_forward(out, d["pool"])
    grads = torch.full((c.T, 64), SENTINEL, dtype=torch.bfloat16, device="cuda")
    c.dfinal.zero_()
    dx, dga, dgx, dd = lib.gated_linear_recurrence_varlen_bwd(
        d["dout"], d["x"], d["ga"], d["gx"], d["decay"], m, d["qsl"], d["slots"], d["has"],
        dgate_a=grads[:, :32].t(), dgate_x=grads[:, 32:].t())
    ref = R.recurrence_grad(c.f, c.z(c.dout), c.z(c.x), c.decay, 8.0, c.bounds)
    for g, name in ((dx, "dx"), (dga, "dgate_a"), (dgx, "dgate_x"), (dd, "ddecay")):
        R.check(g, *ref[name], name)


@pytest.mark.parametrize("layout", ["channel", "token", "strided"])
def test_recurrence_closed_and_open_gates(layout):
    """Gates at and near the ends of their range: a = 1 exactly, a = 0,
    infinite gates; every result finite, as the formulas' limits are."""
    dim, T = 8, 260
    c = Rec([T], dim, "f32", seed=7)
    ends = torch.tensor([NAN, -float("inf"), float("inf"), -200.0, 200.0, -90.0, 60.0, -30.0])
    for ch in range(1, dim):
        c.ga[ch, 40:60] = ends[ch]
        c.gx[ch, 50:70] = -ends[ch]
    c.decay[5], c.decay[6], c.decay[7] = 60.0, -60.0, 3.0
    c.f = R.recurrence(R.f64(c.x), R.f64(c.ga), R.f64(c.gx), c.decay, 8.0, c.bounds)
    d = c.gpu(layout)
    out, m = c.forward(d, layout, states=False)
    # a gate of -60 and less makes a product's exponent range, not its relative
    # error, the limit: compare with the bound of finite moderate gates
    ref = c.f
    assert bool(torch.isfinite(out).all())
    err = (R.f64(out) - ref["h"]).abs()
    assert float((err / (ref["h"].abs() + 1)).max()) < 1e-4
    dx, dga, dgx, dd = lib.gated_linear_recurrence_varlen_bwd(
        d["dout"], d["x"], d["ga"], d["gx"], d["decay"], m, d["qsl"], d["slots"])
    for t in (dx, dga, dgx, dd):
        assert bool(torch.isfinite(t).all())
    want = R.recurrence_grad(ref, R.f64(c.dout), R.f64(c.x), c.decay, 8.0, c.bounds)
    for t, name in ((dx, "dx"), (dga, "dgate_a"), (dgx, "dgate_x")):
        v = want[name][0]
        ok = v.isfinite()
        assert float(((R.f64(t) - v).abs() / (v.abs() + v[ok].abs().mean()))[ok].max()) < 1e-3, name


def test_recurrence_nan_stays_in_its_channel_and_sequence():
    c = Rec([300, 200], 16, "f32", seed=8)
    for layout in ("channel", "token"):
        d = c.gpu(layout)
        base, _ = c.forward(d, layout, states=False)
        d["x"][3, 120] = NAN
        out, _ = c.forward(d, layout, states=False)
        hit = torch.zeros(16, c.T, dtype=torch.bool)
        hit[3, 120:300] = True
        assert bool(out.cpu()[hit].isnan().all())
        assert torch.equal(R.bits(out)[~hit], R.bits(base)[~hit])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,dim", [(1, 1), (3, 7), (8, 512), (65, 130), (300, 64)])
def test_recurrence_update(rows, dim, dtype):
    c = Rec([1] * rows, dim, dtype, seed=rows, inits=range(rows), pads=range(1, rows, 5))
    for odd in (False, True):
        def row(t):
            buf = torch.full((rows, dim + (1 if odd else 8 - dim % 8)), NAN, dtype=t.dtype, device="cuda")
            buf[:, :dim] = t.t()
            return buf[:, :dim]
        pool = c.pool.cuda()
        out = row(torch.full_like(c.x, SENTINEL))
        x = row(c.x)
        lib.gated_linear_recurrence_update(x, row(c.ga), row(c.gx), c.decay.cuda(), pool,
                                           c.slots.cuda(), out=out)
        c.check_forward(out.t(), pool, f"update odd={odd}")
        pool2 = c.pool.cuda()
        lib.gated_linear_recurrence_update(x, row(c.ga), row(c.gx), c.decay.cuda(), pool2,
                                           c.slots.cuda(), out=x)
        live = torch.tensor(c.live)
        assert torch.equal(R.bits(x)[live], R.bits(out)[live])
        assert torch.equal(R.bits(pool), R.bits(pool2))


def test_recurrence_decode_continues_a_prefill():
    """Token by token from the prefill's state: as one longer prefill."""
    c = Rec([150], 64, "f32", seed=11)
    d = c.gpu("token")
    qsl = torch.tensor([0, 140], dtype=torch.int32, device="cuda")
    pool = torch.zeros(1, 64, device="cuda")
    out = torch.empty_like(d["x"])
    lib.gated_linear_recurrence_varlen_fwd(d["x"], d["ga"], d["gx"], d["decay"], pool, qsl, out=out)
    for t in range(140, 150):
        rows = [d[k].t()[t:t + 1] for k in ("x", "ga", "gx")]
        lib.gated_linear_recurrence_update(*rows, d["decay"], pool, out=out.t()[t:t + 1])
    R.check(out, c.f["h"], c.f["eh"], "prefill + decode")
    R.check(pool[0], c.f["last"][0], c.f["elast"][0], "state")


# ---------------------------------------------------------------- conv gradients

@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("W,silu", [(1, True), (2, False), (3, True), (4, True), (4, False)])
def test_conv_gradients(W, silu, dtype, layout):
    n = 4 + LAYOUTS.index(layout)
    lens, dim = [2, 0, 513, 1, 70, 3, 200, 1030][:n], [5, 66, 24, 1, 33][W % 5]
    lead, dt = 1, DT[dtype]
    b = [v + lead for v in R.offsets(lens)]
    T = b[-1] + 2
    pad = 2 if n > 5 else None
    x, g = rand(1, dim, T, dtype=dt), rand(2, dim, T, dtype=dt)
    w, bias = rand(3, dim, W, dtype=dt, scale=0.5), rand(4, dim, dtype=dt)
    has = torch.tensor([k % 2 == 0 for k in range(n)])
    first, end = rand(5, n, dim, W - 1, dtype=dt), rand(6, n, dim, W - 1, dtype=dt)
    slots = torch.randperm(n + 2, generator=torch.Generator().manual_seed(7))[:n].to(torch.int32)
    inside = torch.zeros(T, dtype=torch.bool)
    for k in range(n):
        inside[b[k]:b[k + 1]] = k != pad
    x[:, ~inside], g[:, ~inside] = NAN, NAN
    z = lambda t: R.f64(torch.where(inside, t, torch.zeros_like(t)))  # noqa: E731
    end64 = R.f64(end).clone()
    if pad is not None:
        slots[pad] = -1
        end64[pad] = 0
    gref = z(g)
    ref = R.conv_grad(gref, z(x), R.f64(w), R.f64(bias), b, silu, R.f64(first), end64,
                      R.f64(has.double()))
    pools = [torch.full((n + 2, dim, W - 1), NAN, dtype=dt) for _ in range(2)]
    for k in range(n):
        if k != pad:
            pools[1][int(slots[k])] = end[k]
            if has[k]:
                pools[0][int(slots[k])] = first[k]
    di = torch.full((n + 2, dim, W - 1), SENTINEL, dtype=dt, device="cuda")
    dx = place(torch.full_like(x, SENTINEL), layout)
    _, dw, db = lib.causal_conv1d_varlen_bwd(
        place(g, layout), place(x, layout), w.cuda(), bias.cuda(), pools[0].cuda(),
        torch.tensor(b, dtype=torch.int32, device="cuda"), slots.cuda(), has.cuda(), silu,
        dfinal_states=pools[1].cuda(), dinitial_states=di, dx=dx)
    o = dx.cpu()
    R.check(o[:, inside], ref["dx"][0][:, inside], ref["dx"][1][:, inside], "dx")
    assert bool((o[:, ~inside] == SENTINEL).all()), "dx: wrote outside the sequences"
    R.check(dw, *ref["dweight"], "dweight")
    R.check(db, *ref["dbias"], "dbias")
    d = di.cpu()
    for k in range(n):
        if k != pad:
            R.check(d[int(slots[k])], ref["dinitial"][0][k], ref["dinitial"][1][k], f"dinitial {k}")
            d[int(slots[k])] = SENTINEL
    assert bool((d == SENTINEL).all()), "dinitial: wrote another slot"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens", [[16, 0, 16, 48, 0], [0, 0, 3], [64, 64, 0, 128], [1] * 40, [0, 0],
                                  [100, 2, 1, 0, 1, 1, 60]])
def test_conv_gradients_at_strip_ends(lens, dtype):
    """Rows cut into strips: sequences that end at a cut, are empty there, and
    are shorter than the window; every initial state has a gradient."""
    dim, n, dt = 34, len(lens), DT[dtype]
    b = R.offsets(lens)
    x, g = rand(1, dim, b[-1], dtype=dt), rand(2, dim, b[-1], dtype=dt)
    w, bias = rand(3, dim, 4, dtype=dt, scale=0.5), rand(4, dim, dtype=dt)
    first, end = rand(5, n, dim, 3, dtype=dt), rand(6, n, dim, 3, dtype=dt)
    has = torch.tensor([k % 3 != 1 for k in range(n)])
    ref = R.conv_grad(R.f64(g), R.f64(x), R.f64(w), R.f64(bias), b, True, R.f64(first), R.f64(end),
                      R.f64(has.double()))
    for layout in ("token", "channel"):
        di = torch.empty(n, dim, 3, dtype=dt, device="cuda")
        dx, dw, db = lib.causal_conv1d_varlen_bwd(
            place(g, layout), place(x, layout), w.cuda(), bias.cuda(), first.cuda(),
            torch.tensor(b, dtype=torch.int32, device="cuda"), None, has.cuda(), True,
            dfinal_states=end.cuda(), dinitial_states=di)
        R.check(dx, *ref["dx"], layout + " dx")
        R.check(dw, *ref["dweight"], layout + " dweight")
        R.check(db, *ref["dbias"], layout + " dbias")
        R.check(di, *ref["dinitial"], layout + " dinitial")


@pytest.mark.parametrize("layout", ["channel", "token"])
def test_conv_gradients_plain_call(layout):
    """No bias, no states, a long sequence; equal bits from equal inputs."""
    dim, lens = 130, [3000, 1, 129]
    b = R.offsets(lens)
    x, g, w = rand(1, dim, b[-1]), rand(2, dim, b[-1]), rand(3, dim, 4, scale=0.5)
    ref = R.conv_grad(R.f64(g), R.f64(x), R.f64(w), torch.zeros(dim, dtype=torch.float64), b, True)
    args = (place(g, layout), place(x, layout), w.cuda(), None, None,
            torch.tensor(b, dtype=torch.int32, device="cuda"), None, None, True)
    dx, dw, db = lib.causal_conv1d_varlen_bwd(*args)
    assert db is None
    R.check(dx, *ref["dx"], "dx")
    R.check(dw, *ref["dweight"], "dweight")
    again = lib.causal_conv1d_varlen_bwd(*args)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])


# ---------------------------------------------------------------- norm

DIMS = [1, 7, 64, 130, 1001, 1024, 2056, 4096, 5001, 8192, 20000]


def rows_on_gpu(t, odd):
    rows, dim = t.shape
    buf = torch.full((rows, dim + (1 if odd else 16 - dim % 8)), NAN, dtype=t.dtype, device="cuda")
    buf[:, :dim] = t
    return buf[:, :dim]


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("with_residual", [False, True])
def test_norm_and_gradients(dim, dtype, with_residual):
    dt = DT[dtype]
    rows = 5 if dim > 100 else 67
    x, res = rand(1, rows, dim, dtype=dt), rand(2, rows, dim, dtype=dt, scale=2.0)
    w, g, dres = rand(3, dim, dtype=dt) + 1, rand(4, rows, dim, dtype=dt), rand(5, rows, dim, dtype=dt)
    w = w.to(dt)
    s = R.f64(x) + (R.f64(res) if with_residual else 0)
    y, ey = R.norm(s, R.f64(w), 1e-5)
    # s itself is rounded to fp32 before it is used
    ey = ey + 3 * R.EPS * y.abs()
    for odd in (False, True):
        xd, rd = rows_on_gpu(x, odd), rows_on_gpu(res, odd) if with_residual else None
        out = rows_on_gpu(torch.full_like(x, SENTINEL), odd)
        got = lib.rms_norm_fwd(xd, w.cuda(), 1e-5, residual=rd, out=out)
        R.check(got, y, ey, "out")
        kept = xd
        if with_residual:  # in place: the layer's stream
            R.check(rd, s, R.EPS * s.abs(), "sum")
            kept = rd
            alone = lib.rms_norm_fwd(xd, w.cuda(), 1e-5, residual=rows_on_gpu(res, odd),
                                     residual_out=xd, out=out)
            assert torch.equal(R.bits(alone), R.bits(got)) and torch.equal(R.bits(xd), R.bits(rd))
        ref = R.norm_grad(R.f64(g), R.f64(kept), R.f64(w), 1e-5, R.f64(dres) if with_residual else None)
        gd = rows_on_gpu(g, odd)
        dd = rows_on_gpu(dres, odd) if with_residual else None
        dx, dw = lib.rms_norm_bwd(gd, kept, w.cuda(), 1e-5, dresidual=dd)
        R.check(dx, *ref["dx"], "dx")
        R.check(dw, *ref["dweight"], "dweight")
        dx2, dw2 = lib.rms_norm_bwd(gd, kept, w.cuda(), 1e-5, dresidual=dd, dx=gd)  # in place
        assert torch.equal(R.bits(dx2), R.bits(dx)) and torch.equal(dw, dw2)


@pytest.mark.parametrize("rows", [0, 1, 2, 513, 1500])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm_row_counts(rows, dtype):
    dt, dim = DT[dtype], 136
    x, g, w = rand(1, rows, dim, dtype=dt), rand(2, rows, dim, dtype=dt), rand(3, dim, dtype=dt)
    out = lib.rms_norm_fwd(x.cuda(), w.cuda(), 1e-6)
    y, ey = R.norm(R.f64(x), R.f64(w), 1e-6)
    R.check(out, y, ey, "out")
    dx, dw = lib.rms_norm_bwd(g.cuda(), x.cuda(), w.cuda(), 1e-6)
    ref = R.norm_grad(R.f64(g), R.f64(x), R.f64(w), 1e-6)
    R.check(dx, *ref["dx"], "dx")
    R.check(dw, *ref["dweight"], "dweight")


def check_codes(q, scales, y, ey, group):
    rows, dim = y.shape
    n = dim // group
    amax = y.abs().view(rows, n, group).amax(2)
    eamax = ey.view(rows, n, group).amax(2)
    want = (amax / 448).clamp_min(2.0 ** -126)
    R.check(scales, want, eamax / 448 + 4 * R.EPS * want, "scales")
    sc = R.f64(scales).repeat_interleave(group, 1)
    v = y / sc
    # half a step of e4m3: 2^-4 of a normal value, 2^-10 below 2^-6
    lim = torch.maximum(v.abs() / 16, torch.full_like(v, 2.0 ** -10)) * (1 + 1e-6) + 2 * ey / sc \
        + 4 * R.EPS * v.abs()
    err = (q.cpu().float().double() - v).abs()
    assert bool((err <= lim).all()), float((err - lim).max())


@pytest.mark.parametrize("dim,group", [(1, 0), (7, 0), (64, 32), (192, 64), (1001, 0), (1024, 0),
                                       (1024, 128), (2304, 256), (4096, 0), (4096, 32),
                                       (5056, 64), (8192, 128), (20000, 32), (20001, 0)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm_quant(dim, group, dtype):
    dt, rows = DT[dtype], 9
    x, res = rand(1, rows, dim, dtype=dt), rand(2, rows, dim, dtype=dt, scale=2.0)
    x[3], res[3] = 0, 0                       # a row of zeros
    x[4], res[4] = x[4] * 1e-3, res[4] * 1e-3
    w = (rand(3, dim, dtype=dt) + 1).to(dt)
    s = R.f64(x) + R.f64(res)
    y, ey = R.norm(s, R.f64(w), 1e-5)
    ey = ey + 3 * R.EPS * y.abs()
    for odd in (False, True):
        rd = rows_on_gpu(res, odd)
        q, sc = lib.rms_norm_quant(rows_on_gpu(x, odd), w.cuda(), 1e-5, group_size=group, residual=rd)
        check_codes(q, sc, y, ey, group or dim)
        R.check(rd, s, R.EPS * s.abs(), "sum")
        assert bool((q[3].float() == 0).all())
        # without a residual, into strided outputs
        out = torch.empty(rows, dim + 24, dtype=torch.float8_e4m3fn, device="cuda")[:, :dim]
        q2, sc2 = lib.rms_norm_quant(rd, w.cuda(), 1e-5, group_size=group, out=out)
        y2, ey2 = R.norm(R.f64(rd), R.f64(w), 1e-5)
        check_codes(q2, sc2, y2, ey2, group or dim)


def test_norm_quant_nan_and_huge():
    """A NaN makes its row NaN, and no other row."""
    x = rand(1, 4, 256)
    x[1, 17] = NAN
    x[2] *= 1e15
    for group in (0, 64):
        q, sc = lib.rms_norm_quant(x.cuda(), torch.ones(256, device="cuda"), 0.0, group_size=group)
        assert bool(sc[1].isnan().all()) and bool(q[1].float().isnan().all())
        keep = [0, 2, 3]
        assert bool(sc[keep].isfinite().all()) and bool(q[keep].float().isfinite().all())


# ---------------------------------------------------------------- a layer, graphs, streams

def layer_step(t):
    """norm -> gates -> conv -> recurrence and back, on the library's calls."""
    y = lib.rms_norm_fwd(t["x"], t["nw"], 1e-6, residual=t["res"], residual_out=t["sum"])
    u = y.t()
    pre = u.clone()
    lib.causal_conv1d_varlen_fwd(u, t["cw"], t["cb"], t["cstate"], t["qsl"], None, None, True)
    marks = lib.gated_linear_recurrence_checkpoints(u, t["qsl"])
    out = lib.gated_linear_recurrence_varlen_fwd(u, t["ga"], t["gx"], t["decay"], None, t["qsl"],
                                                 checkpoints=marks)
    du, dga, dgx, dd = lib.gated_linear_recurrence_varlen_bwd(t["dout"], u, t["ga"], t["gx"],
                                                              t["decay"], marks, t["qsl"])
    dc, dw, db = lib.causal_conv1d_varlen_bwd(du, pre, t["cw"], t["cb"], None, t["qsl"], None, None,
                                              True)
    dx, dnw = lib.rms_norm_bwd(dc.t(), t["sum"], t["nw"], 1e-6)
    q, sc = lib.rms_norm_quant(out.t(), t["nw"], 1e-6, group_size=32)
    return dict(out=out, dga=dga, dgx=dgx, dd=dd, dw=dw, db=db, dx=dx, dnw=dnw, q=q, sc=sc)


def layer_inputs(seed, dim=96, lens=(130, 0, 400, 1)):
    b = R.offsets(lens)
    T = b[-1]
    t = dict(x=rand(seed, T, dim), res=rand(seed + 1, T, dim), nw=rand(seed + 2, dim) * 0.1 + 1,
             cw=rand(seed + 3, dim, 4, scale=0.5), cb=rand(seed + 4, dim, scale=0.1),
             ga=rand(seed + 5, dim, T), gx=rand(seed + 6, dim, T), dout=rand(seed + 7, dim, T),
             decay=rand(seed + 8, dim) * 0.3 - 4)
    d = {k: v.cuda() for k, v in t.items()}
    d["sum"] = torch.empty_like(d["x"])
    d["cstate"] = torch.zeros(len(lens), dim, 3, device="cuda")
    d["qsl"] = torch.tensor(b, dtype=torch.int32, device="cuda")
    return t, d, b


def test_layer_runs_together():
    t, d, b = layer_inputs(40)
    got = layer_step(d)
    w = {k: v.double().requires_grad_() for k, v in t.items() if k != "dout"}
    s = w["x"] + w["res"]
    y, _ = R.norm(s, w["nw"], 1e-6)
    outs = []
    for lo, hi in zip(b[:-1], b[1:]):
        u = torch.cat([torch.zeros(96, 3, dtype=torch.float64), y.t()[:, lo:hi]], 1)
        z = w["cb"][:, None] + sum(w["cw"][:, k, None] * u[:, k:k + hi - lo] for k in range(4))
        z = z * torch.sigmoid(z)
        k = 8.0 * torch.nn.functional.softplus(w["decay"])
        la = -k[:, None] * torch.sigmoid(w["ga"][:, lo:hi])
        v = torch.sqrt(-torch.expm1(2 * la)) * torch.sigmoid(w["gx"][:, lo:hi]) * z
        h = torch.zeros(96, dtype=torch.float64)
        for j in range(hi - lo):
            h = torch.exp(la[:, j]) * h + v[:, j]
            outs.append(h)
    out = torch.stack(outs, 1)
    (out * t["dout"].double()).sum().backward()
    # 32-bit results of three operators in a row, of values near one: sums over
    # up to 531 tokens with a memory of about 1 / (1 - a) < 100 tokens keep an
    # error below 100 * 40 units
    for name, ref in (("out", out), ("dga", w["ga"].grad), ("dgx", w["gx"].grad),
                      ("dd", w["decay"].grad), ("dw", w["cw"].grad), ("db", w["cb"].grad),
                      ("dx", w["x"].grad), ("dnw", w["nw"].grad)):
        g = R.f64(got[name])
        scale = float(ref.detach().abs().mean()) + 1e-30
        rel = (g - ref.detach()).abs() / (ref.detach().abs() + scale)
        assert float(rel.max()) < 4000 * R.EPS * 4, (name, float(rel.max()))


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
            for k in d:
                if k not in ("qsl", "sum"):
                    new[k].copy_(d[k]) if k != "cstate" else new[k].zero_()
            side = layer_step(new)
        torch.cuda.synchronize()
        for k in held:
            assert torch.equal(R.bits(replayed[k]), R.bits(eager[k])), (seed, k)
            assert torch.equal(R.bits(side[k]), R.bits(eager[k])), (seed, k, "side stream")


def test_strides_past_32_bits():
    """Rows, channels and slots whose element offsets pass 2^31 and byte offsets
    2^32: planes of one 9 GB buffer."""
    step = (1 << 31) + 8  # elements between two rows (bf16)
    big = torch.empty(2 * step + 4096, dtype=torch.bfloat16, device="cuda")

    def far(shape, at, t=None):
        v = big[at:].as_strided(shape, (step, 1))
        return v if t is None else v.copy_(t)

    bf = dict(dtype=torch.bfloat16)
    x, w = rand(1, 3, 96, **bf), rand(2, 96, **bf)
    y, ey = R.norm(R.f64(x), R.f64(w), 1e-6)
    xd = far((3, 96), 0, x)
    R.check(lib.rms_norm_fwd(xd, w.cuda(), 1e-6, out=far((3, 96), 256)), y, ey, "norm")
    dx, _ = lib.rms_norm_bwd(xd, xd, w.cuda(), 1e-6, dx=far((3, 96), 512))
    R.check(dx, *R.norm_grad(R.f64(x), R.f64(x), R.f64(w), 1e-6)["dx"], "norm dx")
    # three tokens of rows of channels, three channels of tokens
    for rows in (True, False):
        turn = (lambda t: t.t()) if rows else (lambda t: t)
        c = Rec([3] if rows else [100], 96 if rows else 3, "bf16", seed=3)
        c.dfinal.zero_()
        d = c.gpu("token" if rows else "channel")
        shape = (3, 96) if rows else (3, 100)
        d["x"] = turn(far(shape, 1024, turn(c.x)))
        o, m = c.forward(d, None, out=turn(far(shape, 2048).fill_(SENTINEL)))
        c.check_forward(o, d["pool"], "far")
        dx, dga, _, _ = lib.gated_linear_recurrence_varlen_bwd(
            d["dout"], d["x"], d["ga"], d["gx"], d["decay"], m, d["qsl"], d["slots"],
            dx=turn(far(shape, 2560)))
        ref = R.recurrence_grad(c.f, c.z(c.dout), c.z(c.x), c.decay, 8.0, c.bounds)
        R.check(dx, *ref["dx"], "far dx")
        R.check(dga, *ref["dgate_a"], "far dgate_a")
        shape, T = ((3, 64), 3) if rows else ((3, 64), 64)
        dim = 64 if rows else 3
        g, x, w = rand(5, dim, T, **bf), rand(6, dim, T, **bf), rand(7, dim, 4, **bf)
        ref = R.conv_grad(R.f64(g), R.f64(x), R.f64(w), torch.zeros(dim, dtype=torch.float64),
                          [0, T], True)
        q = torch.tensor([0, T], dtype=torch.int32, device="cuda")
        dx, dw, _ = lib.causal_conv1d_varlen_bwd(
            turn(far(shape, 0, turn(g))), turn(far(shape, 256, turn(x))), w.cuda(), None, None, q,
            None, None, True, dx=turn(far(shape, 512)))
        R.check(dx, *ref["dx"], "far conv dx")
        R.check(dw, *ref["dweight"], "far conv dweight")
    # far slots
    c = Rec([1, 1], 96, "f32", seed=4, inits=(0, 1))
    pool = big.view(torch.float32)[40:].as_strided((2, 96), ((1 << 31) - 64, 1)).copy_(c.h0)
    row = lambda t: t.t().contiguous().cuda()  # noqa: E731
    o = lib.gated_linear_recurrence_update(row(c.x), row(c.ga), row(c.gx), c.decay.cuda(), pool)
    R.check(o.t(), c.f["h"], c.f["eh"], "far slots")
    R.check(pool, c.f["last"], c.f["elast"], "far states")


def test_two_streams_and_two_graphs_at_once():
    """Calls in flight on two streams, and two captured graphs replayed in turn
    and side by side, keep their own workspaces."""
    _, d1, _ = layer_inputs(100, lens=(700, 600))
    _, d2, _ = layer_inputs(110, lens=(700, 600))
    want = [{k: v.clone() for k, v in layer_step({**d, "cstate": d["cstate"].clone()}).items()}
            for d in (d1, d2)]
    ins = [{**d, "sum": torch.empty_like(d["sum"]), "cstate": d["cstate"].clone()} for d in (d1, d2)]
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


def test_padded_batch_of_empty_sequences():
    """A fixed batch whose tail has no tokens: states pass through, nothing else
    is touched."""
    for n in (1, 70):  # segments, whole sequences
        lens = [900, 1300] + [0] * n
        for layout in ("token", "channel"):
            c = Rec(lens, 40, "f32", seed=50, inits=range(0, n + 2, 3), pads=range(n, n + 2), trail=9)
            d = c.gpu(layout)
            out, m = c.forward(d, layout)
            c.check_forward(out, d["pool"], layout)
            got, di = c.backward(d, m, layout)
            c.check_backward(got, di, layout)


def test_empty_calls():
    e = dict(dtype=torch.float32, device="cuda")
    q0 = torch.zeros(1, dtype=torch.int32, device="cuda")
    x = torch.empty(5, 0, **e)
    decay = torch.zeros(5, **e)
    lib.gated_linear_recurrence_varlen_fwd(x, x, x, decay, None, q0)
    m = lib.gated_linear_recurrence_checkpoints(x, q0)
    assert bool((lib.gated_linear_recurrence_varlen_bwd(x, x, x, x, decay, m, q0)[3] == 0).all())
    w = torch.ones(5, 4, **e)
    _, dw, db = lib.causal_conv1d_varlen_bwd(x, x, w, decay, None, q0, None, None, True)
    assert bool((dw == 0).all()) and bool((db == 0).all())
    # sequences without tokens: states pass through
    q2 = torch.zeros(3, dtype=torch.int32, device="cuda")
    st = torch.ones(2, 5, **e)
    has = torch.tensor([True, False], device="cuda")
    lib.gated_linear_recurrence_varlen_fwd(x, x, x, decay, st, q2, None, has)
    assert bool((st[0] == 1).all()) and bool((st[1] == 0).all())
    y = torch.empty(0, 5, **e)
    lib.gated_linear_recurrence_update(y, y, y, decay, st)
    assert lib.rms_norm_fwd(y, decay).shape == (0, 5)
