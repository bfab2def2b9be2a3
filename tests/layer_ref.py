"""Plain 64-bit references of the layer operators (gated linear recurrence,
conv gradient, RMS norm), token by token on the CPU, each with a bound on
what fp32 arithmetic may be off by.

A bound counts relative errors in units of EPS = 2^-24 (half a step of
fp32) as they enter: a sigmoid of v is good to |v| + 8 units (the
multiplication by log2 e moves exp's argument by |v| / 2 units, the hardware
exp2 and reciprocal are good to 2 units each), a = exp(-k r) to
4 + (|v| + 12) k r, sqrt(1 - a^2) to |v| + 24 (its own argument's error, at
most doubled by the difference and halved by the root).  ``_units(gates)`` is
the largest of these factors.  The result's own rounding, half a step of its
type, is added by the caller."""
from __future__ import annotations

import numpy as np
import torch

EPS = 2.0 ** -24


def half_step(dtype: torch.dtype) -> float:
    return torch.finfo(dtype).eps / 2


def f64(t):
    return t.detach().cpu().double()


def _units(*gates):
    big = max((float(g.abs()[g.isfinite()].max()) if g.isfinite().any() else 0.0 for g in gates),
              default=0.0)
    return 24.0 + 2.0 * big


def recurrence(x, ga, gx, decay, scale, bounds, h0=None):
    """x, ga, gx [dim, T] f64; h0 [batch, dim].  Returns a dict with h, the
    state before each token, each sequence's last state, and bounds."""
    dim, T = x.shape
    k = scale * torch.nn.functional.softplus(decay.double())
    r, i = torch.sigmoid(ga), torch.sigmoid(gx)
    la = -k[:, None] * r
    a = torch.exp(la)
    m = torch.sqrt(-torch.expm1(2 * la))
    u = m * i * x
    C = EPS * _units(ga, gx) if T else 0.0
    h, before, eh, ebefore = (torch.zeros(dim, T, dtype=torch.float64) for _ in range(4))
    batch = len(bounds) - 1
    last = torch.zeros(batch, dim, dtype=torch.float64) if h0 is None else h0.clone()
    elast = torch.zeros(batch, dim, dtype=torch.float64)
    for b in range(batch):
        s, e = last[b].clone(), torch.zeros(dim, dtype=torch.float64)
        for t in range(bounds[b], bounds[b + 1]):
            before[:, t], ebefore[:, t] = s, e
            e = a[:, t] * e + C * (a[:, t] * s.abs() * (1 - la[:, t]) + u[:, t].abs())
            s = a[:, t] * s + u[:, t]
            h[:, t], eh[:, t] = s, e
        last[b], elast[b] = s, e
    return dict(k=k, r=r, i=i, la=la, a=a, m=m, u=u, h=h, before=before, eh=eh, ebefore=ebefore,
                last=last, elast=elast, C=C)


def recurrence_grad(f, dout, x, decay, scale, bounds, dfinal=None, has=None):
    """Gradients from recurrence()'s result f, each as (value, bound)."""
    dim, T = x.shape
    batch = len(bounds) - 1
    a, la, m, r, i, k, C = (f[n] for n in ("a", "la", "m", "r", "i", "k", "C"))
    dh, edh = torch.zeros(dim, T, dtype=torch.float64), torch.zeros(dim, T, dtype=torch.float64)
    dinit, edinit = (torch.zeros(batch, dim, dtype=torch.float64) for _ in range(2))
    for b in range(batch):
        s = torch.zeros(dim, dtype=torch.float64) if dfinal is None else dfinal[b].clone()
        e = torch.zeros(dim, dtype=torch.float64)
        for t in range(bounds[b + 1] - 1, bounds[b] - 1, -1):
            dh[:, t] = dout[:, t] + s
            edh[:, t] = e + 2 * EPS * (dout[:, t].abs() + s.abs())
            s = a[:, t] * dh[:, t]
            e = a[:, t] * edh[:, t] + C * s.abs() * (1 - la[:, t])
        dinit[b], edinit[b] = s, e
    ix = i * x
    over = torch.where(m > 0, a / m, torch.zeros_like(m)) * ix
    dx, edx = dh * m * i, (edh + 2 * C * dh.abs()) * m * i
    dgx, edgx = dx * x * (1 - i), (edx * x.abs() + C * (dx * x).abs()) * (1 - i) + C * (dx * x).abs() * i
    inner = f["before"] - over
    dlog = a * dh * inner
    edlog = a * (edh * inner.abs() + dh.abs() * (
        f["ebefore"] + 2 * C * (1 - la) * (f["before"].abs() + over.abs())))
    q = k[:, None] * r * (1 - r)
    dga, edga = -q * dlog, q * edlog + C * q * dlog.abs() + C * (k[:, None] * r * r * dlog).abs()
    gain = scale * torch.sigmoid(decay.double())
    terms, eterms = r * dlog, r * edlog + C * (r * dlog).abs()
    # fp32 sums: at most T / 64 + 64 additions behind one another
    ddecay = -gain * terms.sum(1)
    eddecay = gain * (eterms.sum(1) + (T / 64 + 64 + batch) * EPS * terms.abs().sum(1)) + 16 * EPS * ddecay.abs()
    if has is not None:
        dinit, edinit = dinit * has[:, None], edinit * has[:, None]
    return dict(dx=(dx, edx), dgate_a=(dga, edga), dgate_x=(dgx, edgx), ddecay=(ddecay, eddecay),
                dinitial=(dinit, edinit))


def _silu(z):
    return z * torch.sigmoid(z)


def conv(x, w, bias, bounds, silu, first=None):
    """Values of the varlen conv [dim, T]; first [batch, dim, W-1]."""
    dim, T = x.shape
    W = w.shape[1]
    out = torch.zeros(dim, T, dtype=torch.float64)
    for b in range(len(bounds) - 1):
        lo, hi = bounds[b], bounds[b + 1]
        head = first[b] if first is not None else torch.zeros(dim, W - 1, dtype=torch.float64)
        u = torch.cat([head, x[:, lo:hi]], 1)
        z = bias[:, None] + sum(w[:, k, None] * u[:, k:k + hi - lo] for k in range(W))
        out[:, lo:hi] = _silu(z) if silu else z
    return out


def conv_grad(dout, x, w, bias, bounds, silu, first=None, dfinal=None, has=None):
    dim, T = x.shape
    W = w.shape[1]
    batch = len(bounds) - 1
    z2 = lambda *s: torch.zeros(*s, dtype=torch.float64)  # noqa: E731
    dx, edx = z2(dim, T), z2(dim, T)
    dw, edw, db, edb = z2(dim, W), z2(dim, W), z2(dim), z2(dim)
    di, edi = z2(batch, dim, W - 1), z2(batch, dim, W - 1)
    for b in range(batch):
        lo, hi = bounds[b], bounds[b + 1]
        n = hi - lo
        head = first[b] if first is not None else z2(dim, W - 1)
        if has is not None:
            head = head * has[b]
        u = torch.cat([head, x[:, lo:hi]], 1)
        z = bias[:, None] + sum(w[:, k, None] * u[:, k:k + n] for k in range(W))
        az = bias.abs()[:, None] + sum((w[:, k, None] * u[:, k:k + n]).abs() for k in range(W))
        g = dout[:, lo:hi]
        if silu:
            s = torch.sigmoid(z)
            dz = g * s * (1 + z * (1 - s))
            # |silu''| <= 1/2; the factors are good to |z| + 16 units each
            edz = g.abs() * (0.5 * (W + 2) * EPS * az + EPS * (16 + z.abs()) * (s + (s * z * (1 - s)).abs() + (s * s * z).abs()))
        else:
            dz, edz = g, torch.zeros_like(g)
        du, edu = z2(dim, n + W - 1), z2(dim, n + W - 1)
        adu = z2(dim, n + W - 1)
        if dfinal is not None:
            du[:, n:] += dfinal[b]
            adu[:, n:] += dfinal[b].abs()
        for k in range(W):
            du[:, k:k + n] += w[:, k, None] * dz
            edu[:, k:k + n] += w[:, k, None].abs() * edz
            adu[:, k:k + n] += (w[:, k, None] * dz).abs()
            dw[:, k] += (dz * u[:, k:k + n]).sum(1)
            edw[:, k] += (edz * u[:, k:k + n].abs()).sum(1) + (n / 64 + 64 + batch) * EPS * (dz * u[:, k:k + n]).abs().sum(1)
        edu += (W + 1) * EPS * adu
        db += dz.sum(1)
        edb += edz.sum(1) + (n / 64 + 64 + batch) * EPS * dz.abs().sum(1)
        dx[:, lo:hi], edx[:, lo:hi] = du[:, W - 1:], edu[:, W - 1:]
        keep = 1.0 if has is None else float(has[b])
        di[b], edi[b] = du[:, :W - 1] * keep, edu[:, :W - 1] * keep
    return dict(dx=(dx, edx), dweight=(dw, edw), dbias=(db, edb), dinitial=(di, edi))


def norm_units(dim):
    """Relative error of rsqrt(mean(s^2) + eps), in EPS: at most dim / 64 + 10
    additions behind one another (halved by the root), products, division,
    root."""
    return (dim / 64 + 10) / 2 + 8


def norm(s, w, eps):
    y = s * w / torch.sqrt(s.square().mean(1, keepdim=True) + eps)
    return y, (norm_units(s.shape[1]) + 3) * EPS * y.abs()


def norm_grad(dout, x, w, eps, dres=None):
    dim = x.shape[1]
    rstd = 1 / torch.sqrt(x.square().mean(1, keepdim=True) + eps)
    hat, wg = x * rstd, w * dout
    proj = (wg * hat).mean(1, keepdim=True)
    aproj = (wg * hat).abs().mean(1, keepdim=True)
    dx = rstd * (wg - hat * proj)
    U = norm_units(dim) * EPS
    edx = rstd * (8 * EPS * wg.abs() + hat.abs() * (2 * U + (dim / 64 + 14) * EPS) * aproj) + U * dx.abs()
    if dres is not None:
        dx, edx = dx + dres, edx + 2 * EPS * (dx.abs() + dres.abs())
    rows = x.shape[0]
    dw = (dout * hat).sum(0)
    # one row's product is off by U; then at most rows additions
    edw = ((U + 2 * EPS) + rows * EPS) * (dout * hat).abs().sum(0)
    return dict(dx=(dx, edx), dweight=(dw, edw))


def check(got, ref, bound, what):
    """|got - ref| <= bound + half a step of got's type, everywhere."""
    g = f64(got)
    h = half_step(got.dtype)
    # smallest normal step: results below the normal range round by it
    lim = bound + h * (ref.abs() + bound) * (1 + 1e-9) + torch.finfo(got.dtype).tiny
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    bad = ~((g - ref).abs() <= lim)
    if bad.any():
        idx = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())}/{bad.numel()} off; first at {idx}: got "
                             f"{float(g[idx])!r} want {float(ref[idx])!r} within "
                             f"{float(lim[idx]):.3g}")


def bits(t):
    t = t.detach().cpu().contiguous()
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32, 8: torch.int64}[t.element_size()])


def offsets(lens):
    return [0] + [int(v) for v in np.cumsum(lens)]
