"""Layer norm on the GPU where its mean is hard: rows whose values are far from
zero and near each other, in every form of the kernels."""
from __future__ import annotations

import pytest
import torch

import depthwise_causal_conv1d_amd as lib
from tests import layer_ref as R

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def rand(seed, *shape, dtype=torch.float32, scale=1.0):
    t = torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale
    return t.to(dtype)


def statistics(s, eps):
    """d = s - mean and rstd in 64 bits, and what kernels may be off by: a sum of
    dim terms over at most 1024 lanes is (dim / 64 + 10) EPS of its terms off, so a
    first mean by that of |s|; the differences from it are exact to half a step,
    and their own mean, which is then taken out, is off by the same share of them."""
    dim = s.shape[1]
    chain = (dim / 64 + 10) * R.EPS
    mean = s.mean(1, keepdim=True)
    d = s - mean
    first = chain * s.abs().mean(1, keepdim=True) + 2 * R.EPS * mean.abs()
    size = d.abs() + first
    ed = chain * size.mean(1, keepdim=True) + 4 * R.EPS * size
    var = d.square().mean(1, keepdim=True)
    # sum d^2 - (sum d)^2 / n, each a share off
    evar = (3 * chain + 4 * R.EPS) * (size.square().mean(1, keepdim=True))
    rstd = 1 / torch.sqrt(var + eps)
    return d, rstd, ed, evar / (var + eps) + 6 * R.EPS


def on_gpu(t, odd):
    rows, dim = t.shape
    if not odd:
        return t.cuda()
    buf = torch.empty(rows * (dim + 1) + 1, dtype=t.dtype, device="cuda")
    return buf[1:].as_strided((rows, dim), (dim + 1, 1), 1).copy_(t)


def check(x, eps, odd):
    rows, dim = x.shape
    dt = x.dtype
    w, b = (rand(3, dim) * 0.2 + 1).to(dt), rand(4, dim, dtype=dt)
    s, W, B = R.f64(x), R.f64(w), R.f64(b)
    d, rstd, ed, er = statistics(s, eps)
    hat = d * rstd
    ehat = ed * rstd + hat.abs() * er + 2 * R.EPS * (hat.abs() + ed * rstd)
    y = hat * W + B
    out = lib.layer_norm_fwd(on_gpu(x, odd), w.cuda(), b.cuda(), eps, out=on_gpu(x, odd))
    R.check(out, y, ehat * W.abs() + 3 * R.EPS * (y.abs() + ehat * W.abs()), "out")
    g = rand(5, rows, dim, dtype=dt)
    G = R.f64(g)
    wg = G * W
    chain = (dim / 64 + 10) * R.EPS
    flat, proj = wg.mean(1, keepdim=True), (wg * hat).mean(1, keepdim=True)
    eflat = (chain + 3 * R.EPS) * wg.abs().mean(1, keepdim=True)
    eproj = (wg.abs() * ehat).mean(1, keepdim=True) \
        + (2 * chain + 6 * R.EPS) * (wg.abs() * (hat.abs() + ehat)).mean(1, keepdim=True)
    inner = wg - flat - hat * proj
    einner = 4 * R.EPS * (wg.abs() + flat.abs() + (hat * proj).abs()) + eflat \
        + ehat * (proj.abs() + eproj) + hat.abs() * eproj
    edx = rstd * (einner + (inner.abs() + einner) * (er + 3 * R.EPS))
    dx, dw, db = lib.layer_norm_bwd(on_gpu(g, odd), on_gpu(x, odd), w.cuda(), eps, dx=on_gpu(x, odd))
    R.check(dx, rstd * inner, edx, "dx")
    R.check(dw, (G * hat).sum(0), (G.abs() * ehat).sum(0) + rows * R.EPS * (G.abs() * (hat.abs() + ehat)).sum(0),
            "dweight")
    R.check(db, G.sum(0), rows * R.EPS * G.abs().sum(0), "dbias")


# rows of one wave and of four, in vectors and single elements, held and read again
DIMS = [(7, False), (500, True), (1024, False), (1500, True), (4096, False), (5001, True), (8192, False),
        (16384, False), (20001, False)]


@pytest.mark.parametrize("dim,odd", DIMS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_of_one_value(dim, odd, dtype):
    """All channels equal: the normalised row is zero, whatever the sum's rounding."""
    values = torch.tensor([4321.1, -1234.567, 0.1, 3.3e4, -7.7e-3, 0.0, 1e6])
    check(values[:, None].expand(-1, dim).to(DT[dtype]).contiguous(), 1e-5, odd)


@pytest.mark.parametrize("dim,odd", DIMS)
def test_small_differences_far_from_zero(dim, odd):
    """Differences of 2^-4 around 4096.3: the variance and the gradients are theirs."""
    check(4096.3 + rand(1, 6, dim, scale=0.0625), 1e-5, odd)


def test_a_nan_stays_one():
    x = torch.full((3, 700), 4321.1)
    x[1, 5] = float("nan")
    out = lib.layer_norm_fwd(x.cuda(), torch.ones(700, device="cuda"), None, 0.0)
    assert bool(out[1].isnan().all())


@pytest.mark.parametrize("rows,dim", [(1 << 20, 1028), (1 << 18, 8196), ((1 << 20) + 77, 20)])
def test_weights_gradients_of_a_million_equal_rows(rows, dim):
    """Every row the same (strides of zero): a sum of equal terms, whose roundings
    do not cancel.  No fp32 chain is longer than 256 rows: 256 EPS and a few."""
    row, g = rand(1, dim), rand(2, dim).abs() + 0.5
    w = torch.ones(dim)
    hat, rstd, ed, er = statistics(R.f64(row)[None], 1e-5)
    hat = (hat * rstd)[0]
    ehat = (ed * rstd)[0] + hat.abs() * er[0] + 2 * R.EPS * hat.abs()
    wide = lambda t: t.cuda()[None].expand(rows, dim)  # noqa: E731
    dx = torch.empty(rows, dim, device="cuda")
    _, dw, db = lib.layer_norm_bwd(wide(g), wide(row), w.cuda(), 1e-5, dx=dx)
    G, chain = R.f64(g) * rows, 256 * R.EPS
    R.check(db, G, (chain + 8 * R.EPS) * G.abs(), "dbias")
    R.check(dw, G * hat, (chain + 8 * R.EPS) * (G * hat).abs() + G * ehat, "dweight")


@pytest.mark.parametrize("dim,odd", [(64, False), (1000, False), (4096, False), (4095, True), (20001, True)])
@pytest.mark.parametrize("dtype", DT)
def test_equal_channels_whose_squares_overflow(dtype, dim, odd):
    """The differences of equal channels from their rounded mean are 0, or all one
    number of a step of theirs at least, whose square is infinite from 1e28 on: 0
    times weight plus bias either way, and no share in dweight.  dx is the formula's
    with rstd = eps^-1/2 or, where squares are infinite, with 0: finite."""
    x = torch.tensor([2.5e28, 1.1e30, -4.3e33], dtype=torch.float64)[:, None].expand(3, dim).to(DT[dtype])
    w, b, g = rand(1, dim, dtype=DT[dtype]), rand(2, dim, dtype=DT[dtype]), rand(3, 3, dim, dtype=DT[dtype])
    out = lib.layer_norm_fwd(on_gpu(x, odd), w.cuda(), b.cuda(), 1e-5, out=on_gpu(x, odd))
    assert torch.equal(out.cpu(), b.expand(3, dim))
    dx, dw, db = lib.layer_norm_bwd(on_gpu(g, odd), on_gpu(x, odd), w.cuda(), 1e-5, dx=on_gpu(x, odd))
    assert dx.isfinite().all()
    assert torch.equal(dw.cpu(), torch.zeros(dim))
    # three terms
    assert ((db.cpu() - g.double().sum(0)).abs() <= 3 * R.EPS * g.double().abs().sum(0)).all()
