"""The example's 4-bit weights, without a device: what codes, scales and zero points stand for is the weight, for groups of
one sign, equal values and zeros too. A code and a zero point are rounded once each, and the scale, which the code's
distance from the zero point multiplies."""
import os
import sys

import pytest
import torch

from tests.conftest import ROOT

sys.path.insert(0, os.path.join(ROOT, "examples"))
import quantised_layer  # noqa: E402


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_groups_of_every_kind(dtype):
    G, K = quantised_layer.GROUP, 8 * quantised_layer.GROUP
    g = torch.Generator().manual_seed(1)
    w = torch.randn(16, 8, G, generator=g)
    w[:, 1] = w[:, 1].abs() + 3         # one sign, far from zero
    w[:, 2] = -w[:, 2].abs()
    w[:, 3] = 0.5                       # one value
    w[:, 4] = -0.25
    w[:, 5] = 0
    w[:, 6, 1:] = 0                     # one weight
    w[:, 7] *= 1e-3
    layer = quantised_layer.QuantisedLayer(w.view(16, K).to(dtype), torch.ones(K, dtype=dtype))
    q = torch.stack([layer.codes & 15, layer.codes >> 4], dim=2).view(16, 8, G).float()
    z, s = layer.zeros.float()[:, :, None], layer.scales.float()[:, :, None]
    want = w.to(dtype).float()
    span = want.amax(dim=2, keepdim=True).clamp_min(0) - want.amin(dim=2, keepdim=True).clamp_max(0)
    tol = span / 15 * (1 + 15 * torch.finfo(dtype).eps / 2) * (1 + 2 ** -10) + torch.finfo(dtype).tiny
    assert bool(torch.isfinite(s).all()) and bool((layer.zeros <= 15).all())
    assert bool((((q - z) * s - want).abs() <= tol).all())
