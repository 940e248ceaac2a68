"""The gradient norm over the range of its values and of its lengths, against fp64."""
import ctypes
import math

import pytest
import torch

import dropless_moe_expert_gb300 as moe

pytestmark = pytest.mark.gpu
ULP = 2.0 ** -24


@pytest.mark.parametrize("value", [1e18, 2.0 ** -66], ids=str)
def test_sums_of_squares_near_the_ends_of_the_range(value):
    """400 entries in tensors of their own, so in many CTAs: the sum of all squares may pass what fp32 holds (4e38
    here), and the small ones are subnormal (2^-132, exact).  Bound: the square's rounding, the fp64 sum's and the
    root's, then the factor's three and the product's."""
    grads = [torch.full((1,), value, device="cuda") for _ in range(400)]
    ref = 20.0 * float(grads[0])
    clipper = moe.GradClipper(grads, [torch.empty_like(g) for g in grads])
    limit = 0.5 * ref if ref > 1.0 else 1.0
    assert abs(float(clipper(limit)) - ref) <= 4 * ULP * ref
    want = float(grads[0]) * min(1.0, limit / (ref + 1e-6))
    for o in clipper.outs:
        assert abs(float(o) - want) <= 8 * ULP * want
