"""The 64-bit reference of the gated delta rule against automatic
differentiation and differences, and its chunked form (CPU)."""
from __future__ import annotations

import pytest
import torch

from tests import delta_ref as R


def inputs(seed, T, H=2, K=5, V=4):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    q, k = (torch.nn.functional.normalize(r(T, H, K), dim=2) for _ in range(2))
    return q, k, r(T, H, V), -r(T, H).abs() * 0.2, torch.sigmoid(r(T, H)), r(H, K, V), r(T, H, V), r(H, K, V)


@pytest.mark.parametrize("T", [0, 1, 6])
def test_gradients_against_automatic_differentiation(T):
    q, k, v, g, beta, s0, dout, ds = inputs(1, T)
    leaves = [t.clone().requires_grad_() for t in (q, k, v, g, beta, s0)]
    out, states = R.forward(*leaves[:5], 0.7, leaves[5])
    loss = (out * dout).sum() + (states[-1] * ds).sum()
    want = torch.autograd.grad(loss, leaves, allow_unused=True)
    got = R.backward(dout, q, k, v, g, beta, 0.7, states.detach(), ds)
    for name, w in zip(("dq", "dk", "dv", "dg", "dbeta", "dinitial"), want):
        if w is not None:
            assert torch.allclose(got[name], w, rtol=1e-10, atol=1e-12), name


def test_gradients_against_differences():
    args = list(inputs(2, 3))
    dout, ds = args[6], args[7]

    def loss(a):
        out, states = R.forward(*a[:5], 0.7, a[5])
        return float((out * dout).sum() + (states[-1] * ds).sum())

    states = R.forward(*args[:5], 0.7, args[5])[1]
    got = R.backward(dout, *args[:5], 0.7, states, ds)
    for n, name in enumerate(("dq", "dk", "dv", "dg", "dbeta", "dinitial")):
        for at in range(args[n].numel()):
            hi, lo = [t.clone() for t in args], [t.clone() for t in args]
            hi[n].view(-1)[at] += 1e-6
            lo[n].view(-1)[at] -= 1e-6
            # central differences: d^2 in truncation, 1e-16 |loss| / d in rounding
            assert abs((loss(hi) - loss(lo)) / 2e-6 - float(got[name].reshape(-1)[at])) < 1e-7, name


def test_bounds_hold_for_32_bit_arithmetic():
    """The token-by-token form in 32 bits stays within the bounds of the
    chunked one (it has fewer roundings a token, and the same condition), and
    the bounds are small against what they bound."""
    q, k, v, g, beta, s0, dout, ds = inputs(3, 150, H=1, K=16, V=8)
    out, states = R.forward(q, k, v, g, beta, 0.25, s0)
    grads = R.backward(dout, q, k, v, g, beta, 0.25, states, ds)
    low = [t.float() for t in (q, k, v, g, beta, s0, dout, ds)]
    exact = [t.double() for t in low]
    out, states = R.forward(*exact[:5], 0.25, exact[5])
    grads = R.backward(exact[6], *exact[:5], 0.25, states, exact[7])
    b = R.bounds(*exact[:5], 0.25, states, False, grads, exact[6], exact[7])
    out32, states32 = R.forward(*low[:5], 0.25, low[5])
    got = R.backward(low[6], *low[:5], 0.25, states32, low[7])
    assert bool(((out32 - out).abs() <= b["out"]).all())
    assert float(b["out"].max()) < 0.05 * float(out.abs().max())
    for n in ("dq", "dk", "dv", "dg", "dbeta", "dinitial"):
        lim = b[n].unsqueeze(2) if n in ("dq", "dk") else b[n].unsqueeze(1) if n == "dinitial" else b[n]
        assert bool(((got[n] - grads[n]).abs() <= lim).all()), n
        # a bound on dg sums those of a chunk's tokens: its norm is held as well
        assert n == "dg" or float(lim.max()) < 0.05 * float(grads[n].abs().max()), n
        assert R.off(got[n], grads[n]) < R.norm_limit(False), n
