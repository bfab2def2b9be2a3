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
