"""Plain 64-bit reference of the gated delta rule, token by token on the CPU,
and bounds on what the chunked kernels may be off by.

Values come from the definition alone.  A bound follows the chunked form with
norms.  In units: EPS = 2^-24 (half a step of fp32); an fp32 value that enters
a product of bf16 inputs as the sum of two bf16 parts is off by a = 2^-16 of
it (half a step of bf16, twice), with fp32 inputs by nothing (a = 0); a
product over n terms is off by eta(n) = 3 a + (n + 16) EPS of the product of
the norms of its factors (both factors, the small parts' product, n additions,
and exponentials good to 8 EPS of what they multiply, since x e^-x < 1/2).

One chunk, one column v of S, with M = |S0_v|, K and Q spectral norms of the
chunk's keys and queries, T = (I + A)^-1 = I + N, and e-names for bounds:
    eX = |K| (eta M + eS),   eR = beta eX + 4 EPS |R|
    eT = |T|^2 (eta K^2 sqrt(C) + 64 EPS |A|) + a |N| + 64 EPS |T|
    eU = |T| eR + eT |R|
    eS1 = g eS + |K| (eU without its part from eS) + eta |K| |U| + 2 EPS |S1|
The part of eU that comes from eS is no error of its own: the exact chunk
maps S0 to S1 with a norm of at most g = e^(G_C) where 0 <= beta |k|^2 <= 2.
The same for the gradient of the state, from the end.  Sums over columns add
their bounds.  The result's own rounding, half a step of its type, is added
by the caller."""
from __future__ import annotations

import torch

EPS = 2.0 ** -24


def forward(q, k, v, g, beta, scale, s0):
    """One sequence: q, k [T, H, K], v [T, H, V], g, beta [T, H], s0 [H, K, V]
    in 64 bits, q and k of every value head.  Outputs [T, H, V] and the states
    [T + 1, H, K, V] around the tokens."""
    out, states, s = [], [s0], s0
    for t in range(v.shape[0]):
        s = s * torch.exp(g[t])[:, None, None]
        u = beta[t][:, None] * (v[t] - (s * k[t][:, :, None]).sum(1))
        s = s + k[t][:, :, None] * u[:, None, :]
        out.append(scale * (s * q[t][:, :, None]).sum(1))
        states.append(s)
    return (torch.stack(out) if out else v.clone()), torch.stack(states)


def backward(dout, q, k, v, g, beta, scale, states, ds):
    """Gradients of forward() and of the initial state; ds: gradient of the last state."""
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg, db = torch.zeros_like(g), torch.zeros_like(beta)
    marks = [None] * v.shape[0]
    for t in range(v.shape[0] - 1, -1, -1):
        marks[t] = ds  # gradient of the state after token t, from later tokens
        new, alpha = states[t + 1], torch.exp(g[t])[:, None, None]
        old = states[t] * alpha
        dq[t] = scale * (new * dout[t][:, None, :]).sum(2)
        ds = ds + scale * q[t][:, :, None] * dout[t][:, None, :]
        err = v[t] - (old * k[t][:, :, None]).sum(1)
        du = (ds * k[t][:, :, None]).sum(1)
        db[t] = (du * err).sum(1)
        de = beta[t][:, None] * du
        dv[t] = de
        dk[t] = (ds * (beta[t][:, None] * err)[:, None, :]).sum(2) - (old * de[:, None, :]).sum(2)
        ds = ds - k[t][:, :, None] * de[:, None, :]
        dg[t] = (ds * old).sum((1, 2))
        ds = ds * alpha
    return dict(dq=dq, dk=dk, dv=dv, dg=dg, dbeta=db, dinitial=ds, marks=marks)


def _norm(m):
    return torch.linalg.matrix_norm(m, 2)  # over the last two


def bounds(q, k, v, g, beta, scale, states, split, grads=None, dout=None, ds=None):
    """Bounds for every output of forward() and backward() over one sequence:
    a dict of tensors like them ([T, H, ...]; dq and dk one value a token and
    head, that of the whole vector's norm)."""
    C = 64 if split else 32
    a = 2.0 ** -16 if split else 0.0
    T, H, V = v.shape
    K = k.shape[2]
    eta = lambda n: 3 * a + (n + 16) * EPS  # noqa: E731
    one, two, three = eta(K), eta(C), eta(V)
    eS = torch.zeros(H, V, dtype=torch.float64)
    tr = lambda t: t.transpose(0, 1)  # noqa: E731  [c, H, d] -> [H, c, d]
    found = dict(out=torch.zeros_like(v))
    keep = []
    for lo in range(0, T, C):
        hi = min(lo + C, T)
        c = slice(lo, hi)
        kk, qq, vv, b = tr(k[c]), tr(q[c]), tr(v[c]), beta[c].t()
        G = g[c].cumsum(0).t()
        low = torch.ones(hi - lo, hi - lo, dtype=torch.bool).tril()
        e = torch.exp(torch.where(low, G[:, :, None] - G[:, None, :], -torch.inf))
        A = (b[:, :, None] * e * (kk @ kk.transpose(1, 2))).tril(-1)
        eye = torch.eye(hi - lo, dtype=torch.float64)
        Tm = torch.linalg.inv(eye + A)
        P = scale * e * (qq @ kk.transpose(1, 2))
        gam = torch.exp(G)
        S0, S1 = states[lo], states[hi]
        R = b[:, :, None] * (vv - gam[:, :, None] * (kk @ S0))
        U = Tm @ R
        nK, nQ, nT, nP = _norm(kk), _norm(qq), _norm(Tm), _norm(P)
        nA, nN = (torch.linalg.vector_norm(m, dim=(1, 2)) for m in (A, Tm - eye))
        kmax = kk.norm(dim=2).amax(1)
        b1 = b.abs().amax(1)
        M, nR, nU, nS1 = S0.norm(dim=1), R.norm(dim=1), U.norm(dim=1), S1.norm(dim=1)
        x = lambda t: t[:, None]  # noqa: E731
        eT = nT ** 2 * (eta(K) * b1 * kmax ** 2 * (hi - lo) ** 0.5 + 64 * EPS * nA) + a * nN + 64 * EPS * nT
        eRown = x(b1 * nK) * one * M + 4 * EPS * (nR + vv.norm(dim=1))
        eUown = x(nT) * eRown + x(eT) * nR
        eU = eUown + x(nT * b1 * nK) * eS
        qn = qq.norm(dim=2)
        found["out"][c] = tr(
            abs(scale) * qn[:, :, None] * (eS + one * M)[:, None, :]
            + x(nP)[:, :, None] * (eU + two * nU)[:, None, :] + 4 * EPS * (qq @ S0).abs() * abs(scale))
        keep.append((eS, eU, M, nU, nR, U, R, e, gam, b, kk, qq, vv, nK, nQ, nT, nP, nN, eT, G))
        eS = x(gam[:, -1]) * eS + x(nK) * (eUown + two * nU) + 2 * EPS * (nS1 + M)
    found["last"] = eS
    if grads is None:
        return found
    eD = torch.zeros(H, V, dtype=torch.float64)
    for n in ("dq", "dk"):
        found[n] = torch.zeros(T, H, dtype=torch.float64)
    for n in ("dv", "dg", "dbeta"):
        found[n] = torch.zeros_like(grads[n])
    for i in range(len(keep) - 1, -1, -1):
        lo = C * i
        hi = min(lo + C, T)
        c = slice(lo, hi)
        eS, eU, M, nU, nR, U, R, e, gam, b, kk, qq, vv, nK, nQ, nT, nP, nN, eT, G = keep[i]
        x = lambda t: t[:, None]  # noqa: E731
        dS1 = grads["marks"][hi - 1] if hi < T else ds
        dO = tr(dout[c])
        left = torch.exp(G[:, -1:] - G)
        P = scale * e * (qq @ kk.transpose(1, 2))
        A = (b[:, :, None] * e * (kk @ kk.transpose(1, 2))).tril(-1)
        Tm = torch.linalg.inv(torch.eye(hi - lo, dtype=torch.float64) + A)
        dU = P.transpose(1, 2) @ dO + left[:, :, None] * (kk @ dS1)
        dR = Tm.transpose(1, 2) @ dU
        D, nO, ndU, ndR = dS1.norm(dim=1), dO.norm(dim=1), dU.norm(dim=1), dR.norm(dim=1)
        b1 = b.abs().amax(1)
        eUd = two * x(nP) * nO + one * x(nK) * D + 4 * EPS * ndU
        eRown = x(nT) * eUd + x(eT) * ndU
        eR = eRown + x(nT * nK) * eD
        found["dv"][c] = tr(b[:, :, None] * eR[:, None, :] + 4 * EPS * (b[:, :, None] * dR).abs())
        v1 = lambda t: t[:, None, :]  # noqa: E731
        aO, aR, aU = dO.abs(), dR.abs(), U.abs()
        edq = abs(scale) * ((aO * v1(eS + three * M)).sum(2)
                            + x(nK) * ((aO * v1(eU + (three + two) * nU)).sum(2)))
        eZ = (v1(eR * M) + aR * v1(eS + three * M)).sum(2) \
            + x(nK) * (v1(eR * nU) + aR * v1(eU + (three + two) * nU)).sum(2)
        eM = (v1(eU * D) + aU * v1(eD + three * D)).sum(2)
        eW = abs(scale) * x(nQ) * (v1(nO) * ((three + two) * aU + v1(eU))).sum(2) \
            + x(nK * b1) * (v1(eR) * aU + v1(ndR) * (v1(eU) + (three + two) * aU)).sum(2)
        qn, kn = qq.norm(dim=2), kk.norm(dim=2)
        found["dq"][c] = edq.t()
        found["dk"][c] = (eM + eW + b * eZ).t()
        found["dbeta"][c] = ((v1(eR) * vv.abs() + (three + 4 * EPS) * (aR * vv.abs())).sum(2)
                             + kn * (eZ + one * ((aR * v1(M)).sum(2) + x(nK) * (aR * v1(nU)).sum(2)))).t()
        sizes = one * (abs(scale) * qn * ((aO * v1(M + x(nK) * nU)).sum(2))
                       + b * kn * (aR * v1(M + x(nK) * nU)).sum(2) + kn * (aU * v1(D)).sum(2)
                       + kn * (abs(scale) * x(nQ) * (aU * v1(nO)).sum(2)
                               + x(nK * b1) * (aU * v1(ndR)).sum(2)))
        edg = (qn * edq + kn * (b * eZ + eW + eM) + sizes).sum(1) \
            + gam[:, -1] * (eS * D + eD * M + three * M * D).sum(1)
        found["dg"][c] = edg[None, :].expand(hi - lo, H)
        eD = x(gam[:, -1]) * eD + two * x(nQ) * abs(scale) * nO + x(nK * b1) * (two * ndR + eRown) \
            + 2 * EPS * D
    found["dinitial"] = eD
    return found


def norm_limit(split):
    """Of off() for a gradient in fp32: a dozen products between the inputs and
    it, each off by a and, with random signs, sqrt(256) EPS of its result's
    norm; four times that for sums that cancel."""
    return 48 * ((2.0 ** -16 if split else 0.0) + 16 * EPS)


def off(got, ref):
    """Relative error in the 2-norm."""
    return float((got.double() - ref).norm() / ref.norm().clamp_min(1e-300))
