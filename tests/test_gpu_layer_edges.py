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
