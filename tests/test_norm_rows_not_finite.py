"""Rows that are not finite stay alone in every way that rows share the SMs:
teams of warps, pairs of CTAs, a CTA per row, clusters of two CTAs."""
import pytest
import torch

import dropless_moe_expert_gb300 as moe

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32

SHAPES = [(3000, 64, BF16), (3000, 512, BF16), (1000, 640, BF16), (700, 2048, BF16), (400, 4096, F32), (310, 7168, BF16),
          (310, 7168, F32), (400, 5120, BF16), (170, 8256, BF16), (170, 12352, F32), (170, 16384, BF16)]


@pytest.mark.parametrize("T,d,dt", SHAPES, ids=str)
@pytest.mark.parametrize("y,pre", [(True, True), (True, False), (False, True)], ids=["both", "post", "pre"])
def test_rows_that_are_not_finite_stay_alone(T, d, dt, y, pre):
    g = torch.Generator(device="cuda").manual_seed(T + d)

    def normal(*s):
        return torch.randn(*s, generator=g, device="cuda")

    r, out = normal(T, d).to(dt), normal(T, d).to(BF16) if y else None
    dr, dn = normal(T, d).to(dt), normal(T, d).to(BF16) if pre else None
    kw = dict(gamma_post=normal(d) if y else None, gate=normal(T, 1) if y else None, gamma_pre=normal(d) if pre else None)
    fwd = moe.norm_residual(r, out, **kw)
    factors = dict(rstd_post=fwd.rstd_post, rstd_pre=fwd.rstd_pre)
    bwd = moe.norm_residual_backward(fwd.r, dr, dn, out, **kw, **factors)
    bad = [0, 153, T - 1]
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[bad] = False

    def spoilt(t, row, col, value):
        if t is None:
            return None
        t = t.clone()
        t[row, col] = value
        return t

    r2 = spoilt(spoilt(r, 0, 0, float("nan")), T - 1, d - 1, float("-inf"))
    y2 = spoilt(out, 153, d - 1, float("inf"))
    got = moe.norm_residual(r2, y2, **kw)
    for k in ("r", "n", "rstd_post", "rstd_pre"):
        a, b = getattr(got, k), getattr(fwd, k)
        assert (a is None and b is None) or torch.equal(a[keep], b[keep]), k
    if pre:
        assert bool(torch.isnan(got.n[0]).all()) and bool(torch.isnan(got.n[T - 1, d - 1]))
    if y:
        assert bool(torch.isnan(got.r[0, 0])) and not bool(torch.isfinite(got.r[153, d - 1]))

    dr2 = spoilt(spoilt(dr, 0, 0, float("nan")), 153, d - 1, float("inf"))
    dn2 = spoilt(dn, T - 1, d - 1, float("nan"))
    got = moe.norm_residual_backward(fwd.r, dr2, dn2, out, **kw, **factors)
    for k in ("dr", "dy", "dgate"):
        a, b = getattr(got, k), getattr(bwd, k)
        assert (a is None and b is None) or torch.equal(a[keep], b[keep]), k
    assert bool(torch.isnan(got.dr[0, 0])) and not bool(torch.isfinite(got.dr[153, d - 1]))
    if pre:
        assert bool(torch.isnan(got.dr[T - 1]).all())
    if y:
        assert bool(torch.isnan(got.dy[0]).all()) and bool(torch.isnan(got.dgate[0]).all())
        assert bool(torch.isnan(got.dgamma_post[0]))
    assert moe.device_status() == 0
