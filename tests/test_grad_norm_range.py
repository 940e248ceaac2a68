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


@pytest.mark.parametrize("value", [1.4247491, 1.9464883, 1.2040133, 1.0], ids=str)
def test_the_error_does_not_grow_with_the_number_of_elements(value):
    """8.6e9 equal entries (512 times one tensor, which is only read): equal terms round the same way every time,
    so a sum that takes them one after the other drifts.  Bound: a thread's sum of a chunk rounds 18 times, to fp32
    once, the warp's and the block's 21 times, the total 4; half of that after the root, and its rounding."""
    n, times = 1 << 24, 512
    g = torch.full((n,), value, device="cuda")
    norm = torch.zeros(1, device="cuda")
    ws = torch.empty(moe.lib.moe_grad_norm_workspace_size(times), dtype=torch.uint8, device="cuda")
    assert moe.lib.moe_grad_norm((ctypes.c_void_p * times)(*[g.data_ptr()] * times), (ctypes.c_int64 * times)(*[n] * times),
                                 (ctypes.c_int32 * times)(), times, norm.data_ptr(), ws.data_ptr(), ws.numel(),
                                 torch.cuda.current_stream().cuda_stream) == 0
    ref = math.sqrt(n * times) * float(g[0])
    assert abs(float(norm) - ref) <= 24 * ULP * ref
