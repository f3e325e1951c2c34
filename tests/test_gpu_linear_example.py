"""The example of the quantised linear layer, all operators together: its distances from 64-bit arithmetic stay
within what the formats cost. A weight in e4m3 is off by up to 2^-4 of itself, evenly spread that is 2^-4 / sqrt(3)
at the most; with the activations' e4m3 alike, sqrt(2) of that. A 4-bit weight is off by up to half a step of its
group's range / 15, up to 7 standard deviations wide here: 7 / 15 / 2 / sqrt(3) of the weights' spread, and the
zero point's rounding clips at most as much again. The backward pass rounds dy and dx to bfloat16."""
import os
import sys

import pytest
import torch

from tests.conftest import ROOT

sys.path.insert(0, os.path.join(ROOT, "examples"))
import quantised_layer  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [1, 48, 64, 65, 500])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_example(rows, dtype):
    print(f"[linear example] {rows} {dtype}", flush=True)
    got = quantised_layer.run(rows, dtype=dtype, seed=rows)
    e4m3, four_bits = 2 ** 0.5 * 2 ** -4 / 3 ** 0.5, 2 * 7 / 15 / 2 / 3 ** 0.5
    assert got["forward"] <= (four_bits if rows <= quantised_layer.FEW else e4m3)
    if dtype == torch.bfloat16:
        # dy's rounding and dx's, 2^-8 each; dweight adds up dy's
        assert got["dx"] <= 2 * 2.0 ** -8 and got["dweight"] <= 2.0 ** -8
