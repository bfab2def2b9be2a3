"""The gated delta rule on the GPU where its precision is hard: gates that are
nearly closed, many chunks of slow decays, and the walks of full chips."""
from __future__ import annotations

import pytest
import torch

from tests import delta_ref as D
from tests import layer_ref as R
from tests.test_gpu_delta_ops import Case

pytestmark = pytest.mark.gpu


def gate_sizes(c, b=0):
    """|dS| |e^g S| of every token and head of sequence b: dg is their inner
    product, so a share of this is what errors of either may change in it."""
    s = slice(c.bounds[b], c.bounds[b + 1])
    group = c.vh // c.kh
    wide = lambda t: R.f64(t[s]).repeat_interleave(group, 1)  # noqa: E731
    q, k, v, g, beta = wide(c.q), wide(c.k), R.f64(c.v[s]), R.f64(c.g[s]), R.f64(c.beta[s])
    s0 = R.f64(c.h0[b]) * float(c.has[b])
    _, states = D.forward(q, k, v, g, beta, c.scale, s0)
    dout, ds = R.f64(c.dout[s]), R.f64(c.dfinal[b])
    gr = D.backward(dout, q, k, v, g, beta, c.scale, states, ds)
    size = torch.zeros_like(g)
    for t in range(v.shape[0]):
        after = gr["marks"][t] + c.scale * q[t][:, :, None] * dout[t][:, None, :]
        # of the sums that make up the gradient before token t writes: both its terms
        taken = k[t][:, :, None] * gr["dv"][t][:, None, :]
        old = states[t] * torch.exp(g[t])[:, None, None]
        size[t] = (after.norm(dim=(1, 2)) + taken.norm(dim=(1, 2))) * old.norm(dim=(1, 2))
    return size, gr["dg"]


@pytest.mark.parametrize("shape", [(1, 1, 128, 128), (1, 2, 64, 48), (2, 2, 40, 136)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradients_of_nearly_closed_gates(dtype, shape):
    """A gate's gradient has its own size, e^g, whatever the others' is: of tokens at
    tiles' and chunks' ends too, and of two such gates in one tile."""
    c = Case([150], *shape, dtype, seed=31, inits=(0,), rate=0.05)
    for t, g in ((0, -10.0), (5, -12.0), (15, -16.0), (16, -20.0), (31, -14.0), (32, -30.0), (40, -60.0),
                 (41, -25.0), (63, -12.0), (64, -18.0), (80, -8.0), (100, -90.0), (127, -16.0), (149, -40.0)):
        c.g[t] = g
    d = c.gpu()
    _, m = c.forward(d)
    got, _ = c.backward(d, m)
    size, want = gate_sizes(c)
    # a product of a dozen in a row and of a chunk's sums, as norm_limit() counts them;
    # results below the normal range of fp32 may be zero
    lim = D.norm_limit(c.split) * size + 2.0 ** -126
    off = (R.f64(got["dg"]) - want).abs()
    bad = (off > lim).nonzero()
    assert not len(bad), [(int(t), int(h), float(c.g[t, h]), float(off[t, h]), float(want[t, h]), float(lim[t, h]))
                          for t, h in bad[:4]]


def off(got, want):
    """Relative error in the 2-norm."""
    return float((got.double() - want).norm() / want.norm())


def in_64_bits(c, grads=False):
    """Outputs of c's one sequence from the definition in 64 bits on the GPU, token
    by token; with gradients too, the states kept at every 64th token."""
    group = c.vh // c.kh
    f = lambda t: t.cuda().double()  # noqa: E731
    q, k = (f(t).repeat_interleave(group, 1) for t in (c.q, c.k))
    v, g, beta, dout = (f(t) for t in (c.v, c.g, c.beta, c.dout))

    def step(s, t):
        old = s * torch.exp(g[t])[:, None, None]
        err = v[t] - (old * k[t][:, :, None]).sum(1)
        new = old + k[t][:, :, None] * (beta[t][:, None] * err)[:, None, :]
        return old, err, new

    s = f(c.h0[0]) * float(c.has[0])
    out, marks = torch.empty_like(v), []
    for t in range(c.T):
        if t % 64 == 0:
            marks.append(s)
        s = step(s, t)[2]
        out[t] = c.scale * (s * q[t][:, :, None]).sum(1)
    got = dict(out=out, last=s)
    if not grads:
        return got
    ds = f(c.dfinal[0])
    dq, dk, dv, dg, db = (torch.empty_like(t) for t in (q, k, v, g, beta))
    for m in range(len(marks) - 1, -1, -1):
        lo, hi, s, kept = 64 * m, min(64 * m + 64, c.T), marks[m], []
        for t in range(lo, hi):
            kept.append(step(s, t))
            s = kept[-1][2]
        for t in range(hi - 1, lo - 1, -1):
            old, err, new = kept[t - lo]
            dq[t] = c.scale * (new * dout[t][:, None, :]).sum(2)
            ds = ds + c.scale * q[t][:, :, None] * dout[t][:, None, :]
            du = (ds * k[t][:, :, None]).sum(1)
            db[t] = (du * err).sum(1)
            dv[t] = beta[t][:, None] * du
            dk[t] = (ds * (beta[t][:, None] * err)[:, None, :]).sum(2) - (old * dv[t][:, None, :]).sum(2)
            ds = ds - k[t][:, :, None] * dv[t][:, None, :]
            dg[t] = (ds * old).sum((1, 2))
            ds = ds * torch.exp(g[t])[:, None, None]
    pair = lambda t: t.unflatten(1, (c.kh, group)).sum(2)  # noqa: E731
    return got | dict(dq=pair(dq), dk=pair(dk), dv=dv, dg=dg, dbeta=db, dinitial=ds * float(c.has[0]))


# In norms, of sums of many terms of either sign: a value that enters a product rounded to
# half a step e is off by e / 3 in the root mean square, of three factors so rounded and
# fp32 sums of 128 and 64 terms (sqrt(128) EPS / 2) each.  Operands of 22 bits or more: e is
# 2^-22.  A state of decays of 0.999 adds up what some 1000 tokens' chunks (16 of 64) left in
# it at random: four times as much.  Twice that for gradients, behind two walks.
VALUES = (3 * 2.0 ** -22 / 3) + 6 * D.EPS
LONG = [("bf16", 1, 2, 128, 128), ("bf16", 1, 1, 64, 40), ("f32", 1, 1, 128, 77)]


@pytest.mark.parametrize("dtype,kh,vh,K,V", LONG)
@pytest.mark.parametrize("decay", [0.999, 0.99])
def test_states_of_many_chunks_keep_32_bits(dtype, kh, vh, K, V, decay):
    """4096 tokens of slow decays: what a state is off by is that of fp32 sums, not of
    what operands leave out of it (two bf16 parts of each: 2e-6)."""
    c = Case([4096], kh, vh, K, V, dtype, seed=33, inits=(0,), rate=0.0)
    c.g[:] = torch.log(torch.tensor(decay))
    d = c.gpu()
    out, _ = c.forward(d, marks=False)
    want = in_64_bits(c)
    assert off(d["pool"][int(c.slots[0])], want["last"]) < 4 * VALUES
    assert off(out, want["out"]) < 4 * VALUES + R.half_step(out.dtype)
    if dtype == "bf16":
        # one output in 2000 rounds to the other neighbour: an error e moves a share of
        # e / 2^-8 of the values by a step, 2^-7 to 2^-8 of them (two parts: 1.1e-4)
        assert off(out, want["out"].bfloat16().double()) < (4 * VALUES / 2.0 ** -8) ** 0.5 * 2.0 ** -8


@pytest.mark.parametrize("where", ["q", "k", "v", "g", "beta"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_an_infinite_input_spoils_no_value_silently(dtype, where):
    """Every output ahead of an infinite (or huge) input, and beside an infinite q, is
    what it is without it, or not finite; sequences and value heads that do not read it
    keep their bits."""
    c = Case([100, 90], 1, 2, 64, 48, dtype, seed=35, inits=(0, 1))
    d = c.gpu()
    clean, m = c.forward(d)
    keep = d["pool"].clone()
    c2 = Case([100, 90], 1, 2, 64, 48, dtype, seed=35, inits=(0, 1))
    at = getattr(c2, where)
    spot = (70, 0, 5) if at.dim() == 3 else (70, 0)
    at[spot] = -1e38 if where == "beta" else float("inf")
    if where == "g":
        at[spot] = float("nan")
    d2 = c2.gpu()
    out, _ = c2.forward(d2)
    assert torch.equal(R.bits(out[100:]), R.bits(clean[100:]))
    other = 1 if where in ("v", "g", "beta") else None
    if other is not None:
        assert torch.equal(R.bits(out[:, other]), R.bits(clean[:, other]))
    # a value beside it may be rounded with it: by a share of the row that it is in
    fine = out.isfinite()
    near = (out.float() - clean.float()).abs() <= 2.0 ** -6 * clean.float().abs().amax(2, keepdim=True)
    before = torch.zeros_like(fine)
    before[:70] = True  # tokens ahead of it see nothing of it
    assert bool((near | ~fine)[before].all())
    if where == "q":  # it enters one token's output alone
        assert bool((near | ~fine).all())
        assert torch.equal(R.bits(d2["pool"][c2.slots[0].long()]), R.bits(keep[c.slots[0].long()]))
    if where != "beta":  # -1e38 is finite, and so may what it makes be
        assert not bool(out[70, 0].isfinite().all())


@pytest.mark.parametrize("dtype,kh,vh,K,V", LONG + [("bf16", 1, 2, 128, 72), ("bf16", 1, 1, 64, 136)])
@pytest.mark.parametrize("decay", [0.999, 0.9])
def test_gradients_of_many_chunks_keep_32_bits(dtype, kh, vh, K, V, decay):
    """fp32 gradients of gates, betas and states over 1500 tokens: behind two walks,
    twice what values are off by, and a state's four times as above."""
    c = Case([1500], kh, vh, K, V, dtype, seed=37, inits=(0,), rate=0.0)
    c.g[:] = torch.log(torch.tensor(decay))
    d = c.gpu()
    _, m = c.forward(d)
    got, di = c.backward(d, m)
    want = in_64_bits(c, grads=True)
    for n in ("dg", "dbeta"):
        assert off(got[n], want[n]) < 2 * VALUES, n
    assert off(di[int(c.slots[0])], want["dinitial"]) < 4 * VALUES
    for n in ("dq", "dk", "dv"):
        assert off(got[n], want[n]) < 4 * VALUES + R.half_step(got[n].dtype), n


def lengths(n):
    """n sequences, most of a few tokens: around a chunk and its tiles, one empty."""
    few = [1, 65, 17, 3, 64, 0, 130, 16, 33, 5]
    return [few[i] if i < len(few) else 1 + i % 7 for i in range(n)]


@pytest.mark.parametrize("layout", ["dense", "columns"])
@pytest.mark.parametrize("n,kh,vh,K,V", [(33, 4, 8, 128, 128), (33, 2, 4, 77, 129), (17, 8, 8, 64, 136),
                                         (40, 1, 4, 40, 72)])
def test_walks_of_full_chips(n, kh, vh, K, V, layout):
    """Enough workgroups for eight computing waves each (more than 256 of 64 columns), aligned
    rows and others, both widths of K: against the reference, and bit for bit what
    calls of two sequences, which take the other form, give."""
    assert n * vh * -(-V // 64) > 256
    c = Case(lengths(n), kh, vh, K, V, "bf16", seed=41, inits=range(0, n, 3), pads=(3,), trail=3)
    d = c.gpu(layout)
    out, m = c.forward(d, layout)
    got, di = c.backward(d, m, layout)
    some = Case.__new__(Case)
    some.__dict__.update(c.__dict__)
    some.live = [alive and b in (0, 2, 6, 8) for b, alive in enumerate(c.live)]
    pool = d["pool"].cpu()
    for b, s, v, e in some.ref():
        slot = int(c.slots[b])
        R.check(out[s], v["out"], e["out"], f"out {b}")
        R.check(pool[slot], v["last"], e["last"][:, None].expand_as(v["last"]), f"state {b}")
        R.check(di[slot], v["dinitial"], e["dinitial"][:, None].expand_as(v["dinitial"]), f"dinitial {b}")
        for name, t in got.items():
            R.check(t[s], v[name], e[name], f"{name} {b}")
    same = lambda x, y: torch.equal(R.bits(x), R.bits(y))  # noqa: E731
    for b in range(0, n - 1, 2):
        two = Case.__new__(Case)
        two.__dict__.update(c.__dict__)
        lo, hi = c.bounds[b], c.bounds[b + 2]
        two.lens, two.live, two.T = c.lens[b:b + 2], c.live[b:b + 2], hi - lo
        two.slots, two.dfinal = c.slots[b:b + 2], c.dfinal[b:b + 2]
        for t in ("q", "k", "v", "dout"):
            setattr(two, t, getattr(c, t)[lo:hi])
        part = {t: d[t][lo:hi] for t in ("q", "k", "v", "dout", "g", "beta")}
        part |= dict(pool=c.pool.cuda(), slots=d["slots"][b:b + 2].contiguous(),
                     has=d["has"][b:b + 2].contiguous(),
                     qsl=(d["qsl"][b:b + 3] - lo).to(torch.int32).contiguous())
        out2, m2 = two.forward(part, layout)
        got2, di2 = two.backward(part, m2, layout)
        inside = c.inside[lo:hi].cuda()
        assert same(out[lo:hi][inside], out2[inside]), b
        for name in got:
            assert same(got[name][lo:hi][inside], got2[name][inside]), (b, name)
        for k in (b, b + 1):
            if c.live[k]:
                slot = int(c.slots[k])
                assert same(d["pool"][slot], part["pool"][slot]) and same(di[slot], di2[slot]), k
