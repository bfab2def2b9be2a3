"""Edge calls of the layer operators on the GPU: sizes without elements, ends of
the parameters' range, values next to a rounding's border, the variants that
large calls take, and a layer's calls in flight together."""
from __future__ import annotations

import pytest
import torch

import depthwise_causal_conv1d_amd as lib

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
