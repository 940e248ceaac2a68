"""Checks of stored values against fp64 references with an error bound."""
import numpy as np
import torch

from _helpers import to_np


def bf16(a):
    """fp64 values rounded to bf16 (through fp32: both steps are monotone)."""
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(torch.bfloat16).double().numpy()


def within(t, ref, tol):
    """True where `t` may hold a computed value that lies within tol of ref:
    itself for fp32; for bf16 its rounding, which then lies between the
    roundings of the bound's two ends (rounding is monotone)."""
    got = to_np(t).astype(np.float64)
    lo, hi = np.asarray(ref, np.float64) - tol, np.asarray(ref, np.float64) + tol
    if t.dtype == torch.bfloat16:
        lo, hi = bf16(lo), bf16(hi)
    return (lo <= got) & (got <= hi)


def check_within(t, ref, tol, what=""):
    ok = within(t, ref, tol)
    assert ok.all(), f"{what}: {int((~ok).sum())} of {ok.size} elements beyond the bound"
