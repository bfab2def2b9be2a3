"""The 64-bit references of the layer operators against differences and
automatic differentiation (CPU)."""
from __future__ import annotations

import pytest
import torch

from tests import layer_ref as R


def _rand(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


@pytest.mark.parametrize("lens,with_state", [([5], False), ([1, 0, 4, 3], True)])
def test_recurrence_gradients_against_differences(lens, with_state):
    b = R.offsets(lens)
    dim, T, n = 3, b[-1], len(lens)
    x, ga, gx, g = (_rand(k, dim, T) for k in range(4))
    decay = _rand(4, dim) - 3
    h0 = _rand(5, n, dim) if with_state else torch.zeros(n, dim, dtype=torch.float64)
    end = _rand(6, n, dim)

    def loss(x, ga, gx, decay, h0):
        f = R.recurrence(x, ga, gx, decay, 8.0, b, h0)
        return float((f["h"] * g).sum() + (f["last"] * end).sum())

    f = R.recurrence(x, ga, gx, decay, 8.0, b, h0)
    got = R.recurrence_grad(f, g, x, decay, 8.0, b, end)
    args = [x, ga, gx, decay, h0]
    for k, name in enumerate(("dx", "dgate_a", "dgate_x", "ddecay", "dinitial")):
        ref = got[name][0]
        for at in range(args[k].numel()):
            d = 1e-6
            hi, lo = [t.clone() for t in args], [t.clone() for t in args]
            hi[k].view(-1)[at] += d
            lo[k].view(-1)[at] -= d
            # central differences: d^2 in truncation, 1e-16 |loss| / d in rounding
            assert abs((loss(*hi) - loss(*lo)) / (2 * d) - float(ref.reshape(-1)[at])) < 1e-7


@pytest.mark.parametrize("W,silu", [(1, True), (3, False), (4, True)])
def test_conv_gradients_against_autograd(W, silu):
    lens = [2, 0, 1, 6]
    b = R.offsets(lens)
    dim, n = 3, len(lens)
    x, g = _rand(0, dim, b[-1]).requires_grad_(), _rand(1, dim, b[-1])
    w, bias = _rand(2, dim, W).requires_grad_(), _rand(3, dim).requires_grad_()
    first = _rand(4, n, dim, W - 1).requires_grad_()
    end = _rand(5, n, dim, W - 1)
    has = torch.tensor([1.0, 1.0, 0.0, 1.0], dtype=torch.float64)
    loss = 0
    for k in range(n):
        u = torch.cat([first[k] * has[k], x[:, b[k]:b[k + 1]]], 1)
        z = bias[:, None] + sum(w[:, j, None] * u[:, j:j + lens[k]] for j in range(W))
        loss = loss + ((z * torch.sigmoid(z) if silu else z) * g[:, b[k]:b[k + 1]]).sum()
        loss = loss + (u[:, lens[k]:] * end[k]).sum()
    loss.backward()
    got = R.conv_grad(g, x.detach(), w.detach(), bias.detach(), b, silu, first.detach(), end, has)
    for name, t in (("dx", x), ("dweight", w), ("dbias", bias), ("dinitial", first)):
        torch.testing.assert_close(got[name][0], t.grad, rtol=1e-12, atol=1e-12)


def test_norm_gradients_against_autograd():
    x, g = _rand(0, 4, 9).requires_grad_(), _rand(1, 4, 9)
    w, dres = _rand(2, 9).requires_grad_(), _rand(3, 4, 9)
    y, _ = R.norm(x, w, 1e-3)
    ((y * g).sum() + (x * dres).sum()).backward()
    got = R.norm_grad(g, x.detach(), w.detach(), 1e-3, dres)
    torch.testing.assert_close(got["dx"][0], x.grad, rtol=1e-12, atol=1e-12)
    torch.testing.assert_close(got["dweight"][0], w.grad, rtol=1e-12, atol=1e-12)
