"""Edge calls of the layer operators on the GPU: sizes without elements, ends of
the parameters' range, values next to a rounding's border, the variants that
large calls take, and a layer's calls in flight together."""
from __future__ import annotations

import ctypes

import pytest
import torch

import depthwise_causal_conv1d_amd as lib
from depthwise_causal_conv1d_amd import _lib
from tests import layer_ref as R
from tests.test_gpu_layer_ops import DT, NAN, Rec, check_codes, place, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [False, True])
def test_recurrence_without_channels(rows):
    """No channels, tokens enough for segments: nothing to do."""
    x = torch.empty(1000, 0, device="cuda").t() if rows else torch.empty(0, 1000, device="cuda")
    q = torch.tensor([0, 1000], dtype=torch.int32, device="cuda")
    decay = torch.empty(0, device="cuda")
    marks = lib.gated_linear_recurrence_checkpoints(x, q)
    out = lib.gated_linear_recurrence_varlen_fwd(x, x, x, decay, None, q, checkpoints=marks)
    assert out.shape == (0, 1000)
    grads = lib.gated_linear_recurrence_varlen_bwd(out, x, x, x, decay, marks, q)
    assert [tuple(g.shape) for g in grads] == [(0, 1000)] * 3 + [(0,)]


# ---------------------------------------------------------------- 8-bit codes

def border_values(scale):
    """Values v whose quotient v / scale lies at or next to a border between two
    e4m3 values: the nearest fp32 to border * scale and three steps either side."""
    m = torch.arange(17, 32, 2, dtype=torch.float64) / 16          # between 1, 1.125, ...
    border = torch.cat([m * 2.0 ** e for e in range(-6, 8)])
    v = (border * float(scale)).float()
    return torch.cat([(v.view(torch.int32) + k).view(torch.float32) for k in range(-3, 4)])


@pytest.mark.parametrize("dim,group,odd", [(1024, 0, False), (1001, 0, True), (8192, 32, False),
                                           (4096, 128, False), (4096, 256, False),
                                           (8192, 64, True), (20000, 0, False), (40000, 32, False)])
def test_codes_are_the_quotient_rounded_once(dim, group, odd):
    """code = e4m3(y / scale), the quotient's nearest fp32 rounded to nearest
    even, where y is known to the bit: rows of +-1 have a root-mean-square of
    one, so y is the weight with a sign."""
    g = torch.Generator().manual_seed(dim + group)
    n = dim // (group or dim)
    w = torch.empty(dim)
    for k in range(n):
        part = w[k * dim // n:(k + 1) * dim // n]
        # the ends of the range too, where the quotient's remainder would be denormal
        e = [-100, -82, -81, -9, -3, 0, 5, 100][(k + dim) % 8]
        top = (1 + torch.rand(1, generator=g)) * 2.0 ** e
        scale = top * (torch.tensor(1.0) / torch.tensor(448.0))  # as the kernel, to a step of fp32
        v = border_values(scale)
        part.copy_(v[torch.randint(len(v), (len(part),), generator=g)].clamp(-float(top), float(top)))
        part[int(torch.randint(len(part), (1,), generator=g))] = top
    x = (torch.randint(0, 2, (3, dim), generator=g) * 2 - 1).float()
    xd = torch.empty(3, dim + (1 if odd else 0), device="cuda")[:, :dim].copy_(x)
    q, scales = lib.rms_norm_quant(xd, w.cuda(), 0.0, group_size=group)
    y = (x * w).view(3, n, -1)
    sc = scales.cpu()
    want = y.abs().amax(2).double() / 448
    # a product with the nearest fp32 to 1 / 448: a step of each
    assert bool(((sc.double() - want).abs() <= want * 2.0 ** -23).all())
    codes = (y / sc[:, :, None]).to(torch.float8_e4m3fn).view(3, dim)
    got, want = q.cpu().view(torch.uint8), codes.view(torch.uint8)
    assert torch.equal(got, want), f"{int((got != want).sum())} of {got.numel()} codes"


# ---------------------------------------------------------------- ends of decay's range

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["channel", "token", "strided"])
@pytest.mark.parametrize("lens", [[300, 5], [700, 900]])
def test_recurrence_at_the_ends_of_decay(lens, layout, dtype):
    """decay = -inf keeps the state and takes no input in (a = 1), +inf keeps
    nothing (a = 0); so do finite values past the range in which softplus
    differs from those.  A NaN stays in its channel."""
    ends = [float("-inf"), -3.0e38, -200.0, float("inf"), 3.0e38, 1.0e6, NAN]
    near = [-800.0, -800.0, -800.0, 1.0e6, 1.0e6, 1.0e6, 0.0]  # the same a and m in 64 bits
    c = Rec(lens, 9, dtype, seed=60, inits=(0, 1), gate_scale=1.0)
    c.decay[:7] = torch.tensor(near)
    c.f = R.recurrence(c.z(c.x), c.z(c.ga), c.z(c.gx), c.decay, c.scale, c.bounds, R.f64(c.h0))
    ref = R.recurrence_grad(c.f, c.z(c.dout), c.z(c.x), c.decay, c.scale, c.bounds, R.f64(c.dfinal),
                            R.f64(c.has.double()))
    d = c.gpu(layout)
    d["decay"][:7] = torch.tensor(ends, device="cuda")
    out, m = c.forward(d, layout)
    got, di = c.backward(d, m, layout)
    live = [0, 1, 2, 3, 4, 5, 7, 8]
    o = out.cpu()
    R.check(o[live], c.f["h"][live], c.f["eh"][live], "out")
    slots = c.slots.long()
    R.check(d["pool"].cpu()[slots][:, live], c.f["last"][:, live], c.f["elast"][:, live], "states")
    R.check(di.cpu()[slots][:, live], *(t[:, live] for t in ref["dinitial"]), "dinitial")
    for n in ("dx", "dgate_a", "dgate_x"):
        R.check(got[n].cpu()[live], *(t[live] for t in ref[n]), n)
    R.check(got["ddecay"].cpu()[live], *(t[live] for t in ref["ddecay"]), "ddecay")
    assert bool(o[6].isnan().all()) and bool(got["ddecay"][6].isnan())
    # one token
    pool, slots = c.pool.cuda(), c.slots.cuda()
    first = [d[k].t()[[c.bounds[0], c.bounds[1]]].contiguous() for k in ("x", "ga", "gx")]
    one = lib.gated_linear_recurrence_update(*first, d["decay"], pool, slots)
    R.check(one.t()[live], c.f["h"][live][:, c.bounds[:2]], c.f["eh"][live][:, c.bounds[:2]], "update")
    assert bool(one[:, 6].isnan().all())


@pytest.mark.parametrize("layout", ["channel", "token", "strided"])
@pytest.mark.parametrize("lens", [[700, 40], [1400, 600]])
def test_recurrence_infinite_input_and_state(lens, layout):
    """From an infinite input, or from the start where the initial state is
    infinite, the rest of its sequence in that channel is not finite (infinite or
    NaN); everything else is as without it, to the bit."""
    c = Rec(lens, 8, "f32", seed=61, inits=(0, 1))
    d = c.gpu(layout)
    base, _ = c.forward(d, layout, marks=False)
    base_pool, d["pool"] = d["pool"], c.pool.cuda()
    d["x"][3, 100] = float("inf")
    d["x"][4, lens[0] + 7] = float("-inf")
    d["pool"][int(c.slots[1]), 5] = float("inf")
    out, _ = c.forward(d, layout, marks=False)
    hit = torch.zeros(8, c.T, dtype=torch.bool)
    hit[3, 100:lens[0]] = hit[4, lens[0] + 7:] = hit[5, lens[0]:] = True
    o = out.cpu()
    assert not bool(o[hit].isfinite().any())
    assert torch.equal(R.bits(o)[~hit], R.bits(base)[~hit])
    p, want = d["pool"].cpu(), base_pool.cpu()
    for b, ch in ((0, 3), (1, 4), (1, 5)):
        s = int(c.slots[b])
        assert not bool(p[s, ch].isfinite())
        p[s, ch] = want[s, ch] = 0
    assert torch.equal(R.bits(p), R.bits(want))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["channel", "token", "strided"])
@pytest.mark.parametrize("lens", [[260], [420, 500]])
def test_recurrence_gates_at_their_ends(lens, layout, dtype):
    """Closed, open and infinite gates within the derived bounds.  Below a gate of
    -88 the sigmoid is zero here, so r < 2^-126 counts as zero: that moves m = sqrt(2 k r)
    by `least` at most, a state by as much for each token, and the gradients
    (products of such an m, or of its square over itself, with dh) likewise."""
    c = Rec(lens, 8, dtype, seed=62, inits=range(len(lens)))
    ends = [-float("inf"), float("inf"), -200.0, 200.0, -90.0, 60.0, -30.0]
    for ch, v in enumerate(ends):
        c.ga[ch + 1, 40:60] = v
        c.gx[ch + 1, 50:70] = -v
    c.ga[3, 100:] = -90.0  # closed to the end
    c.decay[5], c.decay[6], c.decay[7] = 60.0, -60.0, 3.0
    start, has = R.f64(c.h0), R.f64(c.has.double())
    c.f = f = R.recurrence(R.f64(c.x), R.f64(c.ga), R.f64(c.gx), c.decay, 8.0, c.bounds, start)
    ref = R.recurrence_grad(f, R.f64(c.dout), R.f64(c.x), c.decay, 8.0, c.bounds, R.f64(c.dfinal), has)
    least = (2 * float(f["k"].max()) * 2.0 ** -126) ** 0.5 * float(c.x.abs().max())
    dh = float(c.dout.abs().sum(1).max() + c.dfinal.abs().max())  # a <= 1
    f["eh"] += c.T * least
    f["elast"] += c.T * least
    for v, e in ref.values():
        e += c.T * least * dh
    d = c.gpu(layout)
    out, m = c.forward(d, layout)
    c.check_forward(out, d["pool"], layout)
    got, di = c.backward(d, m, layout)
    for n in ("dx", "dgate_a", "dgate_x", "ddecay"):
        R.check(got[n].cpu(), *ref[n], n)
    R.check(di.cpu()[c.slots.long()], *ref["dinitial"], "dinitial")


# ---------------------------------------------------------------- long sums

def test_recurrence_ddecay_of_a_long_sequence():
    """Equal terms whose roundings do not cancel, over one sequence of 60000 rows
    among empty ones (a mean too short for segments): within the bound of T / 64 + 64 +
    batch additions behind one another."""
    T, batch = 60000, 301
    k = 8.0 * torch.nn.functional.softplus(torch.tensor(-1.0))
    r, i = torch.sigmoid(torch.tensor(0.5)), torch.sigmoid(torch.tensor(0.25))
    a = torch.exp(-k * r)
    m = torch.sqrt(-torch.expm1(-2 * k * r))
    # gradients whose term of the sum, added to itself T / 8 times, is furthest off
    grid = 1.0 + torch.arange(4096) / 4096
    term = a * grid / (1 - a) * (m * i * 0.75 / (1 - a) - a * i * 0.75 / m) * r
    acc = torch.zeros(4096)
    for _ in range(T // 8):
        acc += term
    worst = (acc.double() / term.double() - T // 8).abs().topk(16).indices
    dim = 16
    one = torch.ones(dim, T)
    x, ga, gx, dout = one * 0.75, one * 0.5, one * 0.25, one * grid[worst][:, None]
    decay = torch.full((dim,), -1.0)
    bounds = [0] + [T] * batch
    f = R.recurrence(R.f64(x), R.f64(ga), R.f64(gx), decay, 8.0, bounds)
    ref = R.recurrence_grad(f, R.f64(dout), R.f64(x), decay, 8.0, bounds)["ddecay"]
    q = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    for layout in ("token", "channel"):
        d = [place(t, layout) for t in (dout, x, ga, gx)]
        marks = lib.gated_linear_recurrence_checkpoints(d[1], q)
        lib.gated_linear_recurrence_varlen_fwd(*d[1:], decay.cuda(), None, q, checkpoints=marks)
        dd = lib.gated_linear_recurrence_varlen_bwd(*d, decay.cuda(), marks, q)[3]
        R.check(dd, *ref, layout)


# ---------------------------------------------------------------- variants of large calls

def some_channels(dim, n=8):
    """The first and last channels and some between: each is computed for itself."""
    return torch.unique(torch.cat([torch.arange(min(n, dim)), torch.arange(max(0, dim - n), dim),
                                   torch.randint(0, dim, (n,), generator=torch.Generator().manual_seed(dim))]))


# Whole sequences in rows, the longest first, in both passes (more than 512
# workgroups, 512 tokens a sequence and more); a wave for each channel of long
# sequences, with the launch held to three workgroups a CU (8192 channels in all
# and more, 2048 tokens a sequence); four and sixteen waves for one.
LARGE = [
    ("token", [512, 700, 3, 900, 0, 640, 1100, 64, 800], 4096),
    ("token_odd", [512, 700, 3, 900, 0, 640, 1100, 64, 800], 4001),
    ("channel", [3000, 1, 4000, 1500], 2048),
    ("channel_odd", [3000, 1, 4000, 1500], 2049),
    ("channel", [2000, 1, 1500], 1024),
    ("channel", [4500], 300),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("which", range(len(LARGE)))
def test_recurrence_in_large_calls(which, dtype):
    layout, lens, dim = LARGE[which]
    dt, n = DT[dtype], len(lens)
    b = R.offsets(lens)
    T = b[-1]
    x, ga, gx, dout = (rand(70 + k, dim, T, dtype=dt) for k in range(4))
    decay = rand(75, dim) * 0.5 - 4
    h0, end = rand(76, n, dim), rand(77, n, dim)
    has = torch.tensor([k % 2 == 0 for k in range(n)])
    d = [place(t, layout) for t in (dout, x, ga, gx)]
    q, states = torch.tensor(b, dtype=torch.int32, device="cuda"), h0.cuda()
    marks = lib.gated_linear_recurrence_checkpoints(d[1], q)
    out = place(torch.full_like(x, NAN), layout)
    lib.gated_linear_recurrence_varlen_fwd(*d[1:], decay.cuda(), states, q, None, has.cuda(),
                                           checkpoints=marks, out=out)
    grads = {k: place(torch.full_like(x, NAN), layout) for k in ("dx", "dgate_a", "dgate_x")}
    di = torch.empty_like(states)
    dd = lib.gated_linear_recurrence_varlen_bwd(
        *d, decay.cuda(), marks, q, None, has.cuda(), dfinal_states=end.cuda(), dinitial_states=di,
        **grads)[3]
    ch = some_channels(dim)
    z = lambda t: R.f64(t[ch])  # noqa: E731
    f = R.recurrence(z(x), z(ga), z(gx), decay[ch], 8.0, b, R.f64(h0[:, ch]) * has[:, None])
    ref = R.recurrence_grad(f, z(dout), z(x), decay[ch], 8.0, b, R.f64(end[:, ch]), R.f64(has.double()))
    R.check(out.cpu()[ch], f["h"], f["eh"], "out")
    R.check(states.cpu()[:, ch], f["last"], f["elast"], "states")
    for k in grads:
        R.check(grads[k].cpu()[ch], *ref[k], k)
    R.check(dd.cpu()[ch], *ref["ddecay"], "ddecay")
    R.check(di.cpu()[:, ch], *ref["dinitial"], "dinitial")
    for t in (out, states, di, dd, *grads.values()):  # every element has been written
        assert bool(torch.isfinite(t).all())


@pytest.mark.parametrize("layout", ["token", "token_odd"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_conv_gradients_in_long_strips(dtype, layout):
    """2^23 elements and more in rows: strips of 64 rows, cut and ended anywhere."""
    dim, lens, dt = 1030, [64, 1, 0, 127, 3000, 2, 64, 4943, 0], DT[dtype]
    b, n = R.offsets(lens), len(lens)
    assert b[-1] * dim >= 1 << 23
    x, g = rand(1, dim, b[-1], dtype=dt), rand(2, dim, b[-1], dtype=dt)
    w, bias = rand(3, dim, 4, dtype=dt, scale=0.5), rand(4, dim, dtype=dt)
    first, end = rand(5, n, dim, 3, dtype=dt), rand(6, n, dim, 3, dtype=dt)
    has = torch.tensor([k % 3 != 1 for k in range(n)])
    di = torch.full((n, dim, 3), NAN, dtype=dt, device="cuda")
    dx = place(torch.full_like(x, NAN), layout)
    _, dw, db = lib.causal_conv1d_varlen_bwd(
        place(g, layout), place(x, layout), w.cuda(), bias.cuda(), first.cuda(),
        torch.tensor(b, dtype=torch.int32, device="cuda"), None, has.cuda(), True,
        dfinal_states=end.cuda(), dinitial_states=di, dx=dx)
    c = some_channels(dim)
    ref = R.conv_grad(R.f64(g[c]), R.f64(x[c]), R.f64(w[c]), R.f64(bias[c]), b, True,
                      R.f64(first[:, c]), R.f64(end[:, c]), R.f64(has.double()))
    R.check(dx.cpu()[c], *ref["dx"], "dx")
    R.check(dw.cpu()[c], *ref["dweight"], "dweight")
    R.check(db.cpu()[c], *ref["dbias"], "dbias")
    R.check(di.cpu()[:, c], *ref["dinitial"], "dinitial")
    for t in (dx, dw, db, di):
        assert bool(torch.isfinite(t).all())


@pytest.mark.parametrize("dim,group", [(136, 0), (1001, 0), (1024, 64), (2048, 128), (4096, 256)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm_of_many_rows(dim, group, dtype):
    """4096 rows and more: many workgroups of one row or four, and in the gradients
    each walks several."""
    rows, dt = 9001 if dim <= 1024 else 4099, DT[dtype]
    x, res, g, dres = (rand(80 + k, rows, dim, dtype=dt).cuda() for k in range(4))
    w = (rand(84, dim) * 0.5 + 1).to(dt).cuda()
    total = torch.empty_like(x)
    out = lib.rms_norm_fwd(x, w, 1e-5, residual=res, residual_out=total)
    s = x.double() + res.double()
    y, ey = R.norm(s, w.double(), 1e-5)
    ey = ey + 3 * R.EPS * y.abs()  # s itself is rounded to fp32 before it is used
    near = lambda t, v, e, what: R.check(t, v.cpu(), e.cpu(), what)  # noqa: E731
    near(out, y, ey, "out")
    near(total, s, R.EPS * s.abs(), "sum")
    q, scales = lib.rms_norm_quant(x, w, 1e-5, group_size=group, residual=res, residual_out=total)
    check_codes(q, scales, y.cpu(), ey.cpu(), group or dim)
    dx, dw = lib.rms_norm_bwd(g, total, w, 1e-5, dresidual=dres)
    ref = R.norm_grad(g.double(), total.double(), w.double(), 1e-5, dres.double())
    near(dx, *ref["dx"], "dx")
    near(dw, *ref["dweight"], "dweight")


# ---------------------------------------------------------------- a layer's calls together

def layer_inputs(seed, layout, lens):
    """One layer's tensors, every plane in the same layout: rows of tokens (few
    long sequences: segments, whose two launches hand over through a workspace) or
    channel-major."""
    dim, b = 96, R.offsets(lens)
    T = b[-1]
    plane = (lambda k: rand(k, T, dim).cuda().t()) if layout == "token" else (
        lambda k: rand(k, dim, T).cuda())
    return dict(x=rand(seed, T, dim).cuda(), res=rand(seed + 1, T, dim).cuda(),
                nw=(rand(seed + 2, dim) * 0.1 + 1).cuda(), cw=rand(seed + 3, dim, 4, scale=0.5).cuda(),
                cb=rand(seed + 4, dim, scale=0.1).cuda(), ga=plane(seed + 5), gx=plane(seed + 6),
                dout=plane(seed + 7), decay=(rand(seed + 8, dim) * 0.3 - 4).cuda(),
                cstate=torch.zeros(len(lens), dim, 3, device="cuda"),
                qsl=torch.tensor(b, dtype=torch.int32, device="cuda"), rows=layout == "token")


def layer_step(t):
    """norm -> conv -> recurrence and back, on the library's calls; every value that
    passes from one to the next."""
    k = dict(total=torch.empty_like(t["x"]))
    k["y"] = lib.rms_norm_fwd(t["x"], t["nw"], 1e-6, residual=t["res"], residual_out=k["total"])
    k["v"] = k["y"].t() if t["rows"] else k["y"].t().contiguous()
    k["u"] = k["v"].clone()
    lib.causal_conv1d_varlen_fwd(k["u"], t["cw"], t["cb"], t["cstate"], t["qsl"], None, None, True)
    marks = lib.gated_linear_recurrence_checkpoints(k["u"], t["qsl"])
    k["h"] = lib.gated_linear_recurrence_varlen_fwd(k["u"], t["ga"], t["gx"], t["decay"], None, t["qsl"],
                                                    checkpoints=marks)
    k["du"], k["dga"], k["dgx"], k["dd"] = lib.gated_linear_recurrence_varlen_bwd(
        t["dout"], k["u"], t["ga"], t["gx"], t["decay"], marks, t["qsl"])
    k["dv"], k["dcw"], k["dcb"] = lib.causal_conv1d_varlen_bwd(
        k["du"], k["v"], t["cw"], t["cb"], None, t["qsl"], None, None, True)
    k["dy"] = k["dv"].t() if t["rows"] else k["dv"].t().contiguous()
    k["dx"], k["dnw"] = lib.rms_norm_bwd(k["dy"], k["total"], t["nw"], 1e-6)
    k["q"], k["scales"] = lib.rms_norm_quant(k["h"].t().contiguous(), t["nw"], 1e-6, group_size=32)
    return k


LAYERS = [("token", (700, 600)), ("channel", (2500, 1700))]


def assert_forms(t, k, lens):
    """The planes are what the fast forms take, and rows of them are cut into segments."""
    planes = [t["ga"], t["gx"], t["dout"], k["u"], k["h"], k["v"], k["dv"]] + [
        k[n] for n in ("du", "dga", "dgx")]
    fwd, bwd = ctypes.c_int64(), ctypes.c_int64()
    assert _lib.load().gated_linear_recurrence_workspace(
        sum(lens), len(lens), 96, ctypes.byref(fwd), ctypes.byref(bwd)) == 0
    if t["rows"]:
        assert fwd.value > 0 and all(p.stride(0) == 1 for p in planes)
    else:
        assert all(p.stride(1) == 1 for p in planes)


@pytest.mark.parametrize("layout,lens", LAYERS)
def test_each_call_of_a_layer_against_its_reference(layout, lens):
    """Every call's results within its own derived bound, at the values that the
    call before left."""
    t = layer_inputs(200, layout, lens)
    k = layer_step(t)
    assert_forms(t, k, lens)
    b, c = R.offsets(lens), {n: R.f64(v) for n, v in {**t, **k}.items()
                             if n not in ("qsl", "rows", "q")}
    s = c["x"] + c["res"]
    y, ey = R.norm(s, c["nw"], 1e-6)
    R.check(k["y"], y, ey + 3 * R.EPS * y.abs(), "norm")
    u = R.conv(c["v"], c["cw"], c["cb"], b, True)
    # four products and sums, then |silu'| < 1.1 and the sigmoid's |z| + 16 units
    z = R.conv(c["v"], c["cw"], c["cb"], b, False)
    az = R.conv(c["v"].abs(), c["cw"].abs(), c["cb"].abs(), b, False)
    R.check(k["u"], u, R.EPS * (6 * 1.1 * az + (16 + z.abs()) * u.abs()), "conv")
    f = R.recurrence(c["u"], c["ga"], c["gx"], t["decay"].cpu(), 8.0, b)
    R.check(k["h"], f["h"], f["eh"], "recurrence")
    ref = R.recurrence_grad(f, c["dout"], c["u"], t["decay"].cpu(), 8.0, b)
    for n, r in (("du", "dx"), ("dga", "dgate_a"), ("dgx", "dgate_x"), ("dd", "ddecay")):
        R.check(k[n], *ref[r], n)
    ref = R.conv_grad(c["du"], c["v"], c["cw"], c["cb"], b, True)
    for n, r in (("dv", "dx"), ("dcw", "dweight"), ("dcb", "dbias")):
        R.check(k[n], *ref[r], n)
    ref = R.norm_grad(c["dy"], c["total"], c["nw"], 1e-6)
    R.check(k["dx"], *ref["dx"], "dx")
    R.check(k["dnw"], *ref["dweight"], "dnw")
    y, ey = R.norm(c["h"].t(), c["nw"], 1e-6)
    check_codes(k["q"], k["scales"], y, ey, 32)


@pytest.mark.parametrize("layout,lens", LAYERS)
def test_layers_in_flight_on_streams_and_in_graphs(layout, lens):
    """Two layers on two streams at once, then two captured graphs replayed one
    after another and side by side, with eager work of a third layer between:
    the bits of each layer alone."""
    lib.sconv_init()
    ins = [layer_inputs(seed, layout, lens) for seed in (300, 310, 320)]
    want = [{n: v.clone() for n, v in layer_step(t).items()} for t in ins]
    assert_forms(ins[0], want[0], lens)

    def same(got, k, what):
        for n in want[k]:
            assert torch.equal(R.bits(got[n]), R.bits(want[k][n])), (k, n, what)

    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for turn in range(4):
        got = [None, None]
        for k in (0, 1):
            with torch.cuda.stream(streams[k]):
                for _ in range(3):
                    got[k] = layer_step(ins[k])
        torch.cuda.synchronize()
        for k in (0, 1):
            same(got[k], k, f"streams, turn {turn}")
    graphs, held = [], []
    for k in (0, 1):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held.append(layer_step(ins[k]))
        graphs.append(g)
    for turn in range(4):
        for k in (0, 1):
            for v in held[k].values():  # what an earlier replay left
                v.zero_()
        torch.cuda.synchronize()
        for k in (0, 1):
            with torch.cuda.stream(streams[k if turn % 2 else 0]):
                graphs[k].replay()
        eager = layer_step(ins[2])
        torch.cuda.synchronize()
        for k in (0, 1):
            same(held[k], k, f"graphs, turn {turn}")
        same(eager, 2, f"eager, turn {turn}")
