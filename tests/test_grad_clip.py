"""GPU parity of the global gradient norm and clipping against fp64.

Bounds.  A thread adds at most ceil(chunks / CTAs) * 40 squares one after the
other, then trees of five and sixteen: with the tests' sizes under 128
roundings of positive terms, so the norm is within 128 * 2^-24 relative (the
square root halves it).  A clipped entry takes the factor (the norm's error and
three roundings) and a product: 160 * 2^-24 relative, before a bf16 rounding
(_bounds.within)."""
import numpy as np
import pytest
import torch

import dropless_moe_expert_gb300 as moe
from oracle import operators as op

from _bounds import check_within
from _helpers import to_np

pytestmark = pytest.mark.gpu
ULP = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16


def _grads(sizes, kinds, seed=0, std=0.1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(std * torch.randn(n, generator=g, device="cuda")).to(k) for n, k in zip(sizes, kinds)]


def _check(grads, outs, norm, max_norm):
    ref = op.grad_norm([to_np(g) for g in grads])
    assert abs(float(norm) - ref) <= 128 * ULP * ref
    c = op.clip_factor(ref, max_norm)
    for g, o in zip(grads, outs):
        want = c * to_np(g).astype(np.float64)
        check_within(o, want, 160 * ULP * np.abs(want) + 1e-40)


CASES = [
    ([1], [F32], 0.01), ([1], [BF16], 0.01), ([7, 0, 1, 33], [F32, BF16, BF16, F32], 0.1),
    ([16384, 16385, 16383], [F32, BF16, F32], 1.0), ([1000003, 5, 4096], [BF16, F32, F32], 2.0),
    ([100] * 600, [F32] * 600, 1.0), ([3 + i % 11 for i in range(1100)], [F32 if i % 2 else BF16 for i in range(1100)], 1.0),
    ([16384 * 400 + 77], [F32], 5.0), ([64] * 512, [BF16] * 512, 0.5), ([64] * 513, [BF16] * 513, 0.5),
]


@pytest.mark.parametrize("sizes,kinds,max_norm", CASES, ids=lambda v: str(v)[:24])
def test_norm_and_clip(sizes, kinds, max_norm):
    grads = _grads(sizes, kinds)
    raw = [g.clone() for g in grads]
    outs = [torch.full_like(g, float("nan")) for g in grads]
    clipper = moe.GradClipper(grads, outs)
    norm = clipper(max_norm).clone()
    _check(raw, outs, norm, max_norm)
    assert all(torch.equal(a, b) for a, b in zip(grads, raw))          # the inputs are only read
    assert torch.equal(clipper(), norm)                                # the norm alone, the same bits
    again = [o.clone() for o in outs]
    assert torch.equal(clipper(max_norm), norm) and all(torch.equal(a, b) for a, b in zip(outs, again))
    in_place = moe.GradClipper(grads)
    assert torch.equal(in_place(max_norm), norm) and all(torch.equal(a, b) for a, b in zip(grads, outs))


def test_views_at_any_alignment():
    """Tensors packed without padding, and outputs aligned otherwise than their inputs."""
    sizes = [5, 1, 30, 17, 40000, 3, 9]
    for kind in (F32, BF16):
        for shift in (0, 1, 3):
            flat = _grads([sum(sizes) + 8], [kind], seed=shift)[0]
            out = torch.full_like(flat, 7.0)
            grads = list(torch.split(flat[2:2 + sum(sizes)], sizes))
            outs = list(torch.split(out[shift:shift + sum(sizes)], sizes))
            norm = moe.GradClipper(grads, outs)(0.5)
            _check(grads, outs, norm, 0.5)
            # nothing beside the outputs was written
            assert bool((out[:shift] == 7.0).all()) and bool((out[shift + sum(sizes):] == 7.0).all())


def test_below_the_limit_nothing_changes():
    grads = _grads([1000, 333], [F32, BF16])
    raw = [g.clone() for g in grads]
    for limit in (1e6, float("inf")):
        norm = moe.GradClipper(grads)(limit)
        assert all(torch.equal(a, b) for a, b in zip(grads, raw))
        outs = [torch.empty_like(g) for g in grads]
        assert torch.equal(moe.GradClipper(grads, outs)(limit), norm)
        assert all(torch.equal(a, b) for a, b in zip(outs, raw))


def test_zeros_and_nothing():
    grads = [torch.zeros(100, device="cuda"), torch.zeros(0, device="cuda")]
    assert float(moe.GradClipper(grads)(1.0)) == 0.0 and not bool(grads[0].any())
    assert float(moe.GradClipper([torch.zeros(0, device="cuda")])(1.0)) == 0.0
    assert float(moe.GradClipper([])(1.0)) == 0.0 and float(moe.GradClipper([])()) == 0.0


def test_values_that_are_not_finite():
    """As the formula: an infinity gives an infinite norm and a factor of zero, a NaN gives NaN."""
    grads = _grads([1000, 50], [F32, BF16])
    grads[1][3] = float("inf")
    outs = [torch.empty_like(g) for g in grads]
    assert float(moe.GradClipper(grads, outs)(1.0)) == float("inf")
    assert not bool(outs[0].any()) and bool(torch.isnan(outs[1][3])) and int(torch.isnan(outs[1]).sum()) == 1
    grads[0][999] = float("nan")
    assert np.isnan(float(moe.GradClipper(grads, outs)(1.0)))
    assert all(bool(torch.isnan(o).all()) for o in outs)


def test_streams_and_graphs():
    grads = _grads([70000, 12345], [F32, BF16])
    outs = [torch.empty_like(g) for g in grads]
    clipper = moe.GradClipper(grads, outs)
    ref = [clipper(0.5).clone()] + [o.clone() for o in outs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        norm = clipper(0.5)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip([norm] + outs, ref))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        clipper(0.5)
    for g in grads:
        g.mul_(2.0)       # the captured calls read the gradients' new values
    graph.replay()
    torch.cuda.synchronize()
    _check(grads, outs, clipper.norm, 0.5)


def test_offsets_past_32_bits():
    n = (1 << 31) + 1003
    g = torch.zeros(n, dtype=BF16, device="cuda")
    g[-1001:] = 2.0
    g[5] = 8.0
    norm = float(moe.GradClipper([g])(1.0))
    ref = np.sqrt(1001 * 4.0 + 64.0)
    assert abs(norm - ref) <= 128 * ULP * ref
    c = op.clip_factor(ref, 1.0)
    check_within(g[-1001:], np.full(1001, 2.0 * c), 160 * ULP * 2.0 * c)
    assert not bool(g[6:-1001].any())
