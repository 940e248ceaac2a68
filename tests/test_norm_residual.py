"""GPU parity of the norms, gate and residual between two layers against
oracle/operators.py (fp64).

Bounds.  A row's sum of d squares adds at most d / 64 terms in one register
(no fewer than 64 threads share a row of more than 4096 columns, 8 a smaller
one) and then a tree: with N = d / 8 + 16 roundings its relative error is
under N 2^-24 (positive terms), half of that after the square root.  u and r'
take five more roundings, so r' is within C 2^-24 of |a r| + |g u| with
C = N + 16, and n within twice that; a bf16 store rounds once more, which
_bounds.within covers exactly.  The
backward's row means have the same N; dr is within 2 C 2^-24 of the sum of its
terms' magnitudes, dy (two means deep) within 4 C 2^-24; the sums over T tokens
add T roundings of theirs."""
import numpy as np
import pytest
import torch

import dropless_moe_expert_gb300 as moe
from oracle import operators as op

from _bounds import check_within
from _helpers import to_np

pytestmark = pytest.mark.gpu
ULP = 2.0 ** -24
FORMS = {"both": (1, 1, 1), "post": (1, 1, 0), "add": (1, 0, 1), "sum": (1, 0, 0), "pre": (0, 0, 1)}  # y, post, pre

# T, d, residual, form, gate, res_scale
CASES = [(1, 7168, torch.float32, "both", "channel", 1.0), (1, 64, torch.bfloat16, "both", "token", 0.5),
         (7, 128, torch.bfloat16, "pre", "none", 1.0), (300, 4096, torch.bfloat16, "both", "channel", 0.5),
         (517, 192, torch.float32, "both", "token", 0.7), (129, 2368, torch.float32, "post", "channel", 1.0),
         (129, 2368, torch.bfloat16, "add", "none", 1.0), (64, 1024, torch.float32, "sum", "token", -1.0),
         (33, 16384, torch.float32, "both", "channel", 1.0), (33, 16384, torch.bfloat16, "both", "none", 1.0),
         (20, 8256, torch.bfloat16, "both", "token", 1.0), (700, 320, torch.bfloat16, "both", "none", 1.0),
         (611, 7168, torch.float32, "both", "token", 1.0), (2, 12352, torch.float32, "pre", "none", 1.0),
         (1000, 2048, torch.bfloat16, "sum", "channel", 0.0), (45, 64, torch.float32, "post", "token", 1.0),
         (1221, 512, torch.bfloat16, "both", "channel", 1.0), (3, 5120, torch.bfloat16, "add", "channel", 1.0),
         (700, 2816, torch.float32, "both", "token", 1.0), (400, 4096, torch.float32, "pre", "none", 1.0),
         (5000, 64, torch.bfloat16, "both", "channel", 1.0), (333, 1536, torch.float32, "both", "channel", 0.5),
         (457, 5120, torch.bfloat16, "both", "token", 1.0), (2600, 256, torch.float32, "post", "token", 1.0),
         (613, 5120, torch.bfloat16, "pre", "none", 1.0), (306, 6144, torch.bfloat16, "post", "channel", 1.0),
         (155, 12288, torch.float32, "sum", "token", 1.0), (310, 5184, torch.float32, "post", "none", 1.0),
         (400, 8256, torch.bfloat16, "both", "channel", 0.5), (170, 16384, torch.float32, "both", "token", 1.0),
         (161, 12352, torch.bfloat16, "post", "channel", 1.0), (239, 16384, torch.bfloat16, "both", "token", 1.0)]


def _case(c, seed=0):
    T, d, dt, form, gate, a = c
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*s):
        return torch.randn(*s, generator=g, device="cuda")

    y, post, pre = FORMS[form]
    r = (3.0 * normal(T, d)).to(dt)
    kw = dict(gamma_post=1 + 0.2 * normal(d) if post else None, gamma_pre=1 + 0.2 * normal(d) if pre else None,
              gate={"none": None, "channel": 0.3 * normal(d), "token": normal(T, 1)}[gate], res_scale=a)
    return r, (0.3 * normal(T, d)).to(torch.bfloat16) if y else None, kw, (normal(T, d).to(dt),
                                                                          normal(T, d).to(torch.bfloat16) if pre else None)


def _np(kw):
    return {k: to_np(v) if isinstance(v, torch.Tensor) else v for k, v in kw.items()}


def _opt(t):
    return None if t is None else to_np(t)


def _c(d):
    return d / 8 + 32


def _check_forward(out, r, y, kw, eps=1e-6):
    x, n, rp, rq, mag = op.norm_residual(to_np(r), _opt(y), eps=eps, **_np(kw))
    C = _c(r.shape[1]) * ULP
    if y is not None:
        check_within(out.r, x, C * mag + 1e-38, "r")
    for got, ref in ((out.rstd_post, rp), (out.rstd_pre, rq)):
        assert (got is None) == (ref is None)
        if ref is not None:
            # rstd_pre moves with the error of r' too: |a r| + |g u| over the row's root mean square
            slack = np.sqrt(np.mean(mag ** 2, axis=1)) * ref if ref is rq else 1.0
            assert np.all(np.abs(to_np(got) - ref) <= C * ref * (1 + slack))
    if n is not None:
        g = np.abs(np.asarray(_np(kw)["gamma_pre"], np.float64))
        row = np.sqrt(np.mean(mag ** 2, axis=1, keepdims=True))
        tol = 2 * C * rq[:, None] * g * (mag + np.abs(x) * (1 + row * rq[:, None]))
        check_within(out.n, n, tol + 1e-38, "n")


def _backward_args(out, kw):
    return dict(kw, rstd_post=out.rstd_post, rstd_pre=out.rstd_pre)


def _check_backward(got, r2, y, dr, dn, args):
    ref = op.norm_residual_backward(to_np(r2), _opt(dr), _opt(dn), _opt(y), **_np(args))
    T, d = r2.shape
    C = _c(d) * ULP
    for name, t, c in (("dr", got.dr, 2 * C), ("dy", got.dy, 4 * C), ("dgamma_pre", got.dgamma_pre, 2 * C + T * ULP),
                       ("dgamma_post", got.dgamma_post, 4 * C + T * ULP), ("dgate", got.dgate, 4 * C + T * ULP)):
        assert (t is not None) == (name in ref), name
        if t is not None:
            value, mag = ref[name]
            assert tuple(t.shape) == value.shape
            check_within(t, value, c * mag + 1e-37, name)


@pytest.mark.parametrize("c", CASES, ids=str)
def test_forward_and_backward(c):
    r, y, kw, (dr, dn) = _case(c)
    out = moe.norm_residual(r, y, **kw)
    _check_forward(out, r, y, kw)
    args = _backward_args(out, kw)
    got = moe.norm_residual_backward(out.r, dr, dn, y, **args)
    _check_backward(got, out.r, y, dr, dn, args)
    again = moe.norm_residual_backward(out.r, dr, dn, y, **args)
    for k, v in vars(got).items():
        if v is not None and k != "workspace" and not k.startswith("_"):
            assert torch.equal(v, vars(again)[k]), k      # a fixed order of addition


@pytest.mark.parametrize("c", [c for c in CASES if c[3] in ("both", "add", "pre")][:6], ids=str)
def test_backward_without_a_stream_gradient(c):
    """The last norm of a model: nothing reads the stream after it."""
    r, y, kw, (_, dn) = _case(c, 1)
    out = moe.norm_residual(r, y, **kw)
    args = _backward_args(out, kw)
    _check_backward(moe.norm_residual_backward(out.r, None, dn, y, **args), out.r, y, None, dn, args)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_in_place_buffers_and_streams(dt):
    """r_out over r and dr over the incoming gradient, reused buffers, another stream, a captured graph: the same bits."""
    c = (203, 1088, dt, "both", "channel", 0.5)
    r, y, kw, (dr, dn) = _case(c)
    ref = moe.norm_residual(r, y, **kw)
    args = _backward_args(ref, kw)
    gref = moe.norm_residual_backward(ref.r, dr, dn, y, **args)
    r_in, dr_in = r.clone(), dr.clone()
    out = moe.NormResidual.empty(203, 1088, dt)
    out.r = r_in
    gout = moe.NormResidualGrads.empty(203, 1088, dt, gate="channel")
    gout.dr = dr_in
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        moe.norm_residual(r_in, y, out=out, **kw)
        moe.norm_residual_backward(ref.r, dr_in, dn, y, out=gout, **args)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()

    def same():
        assert torch.equal(out.r, ref.r) and torch.equal(out.n, ref.n)
        for k in ("dr", "dy", "dgamma_pre", "dgamma_post", "dgate"):
            assert torch.equal(getattr(gout, k), getattr(gref, k)), k

    same()
    r_in.copy_(r)
    dr_in.copy_(dr)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        moe.norm_residual(r_in, y, out=out, **kw)
        moe.norm_residual_backward(ref.r, dr_in, dn, y, out=gout, **args)
    r_in.copy_(r)
    dr_in.copy_(dr)
    out.n.zero_()
    gout.dgate.zero_()
    graph.replay()
    torch.cuda.synchronize()
    same()


def test_rows_of_zeros_and_cancelling_sums():
    """A row of zeros has the factor 1 / sqrt(eps); a stream that the output cancels stays finite."""
    T, d = 5, 256
    r = torch.zeros(T, d, device="cuda")
    y = torch.zeros(T, d, device="cuda", dtype=torch.bfloat16)
    r[3] = 1.0
    y[3] = -1.0
    y[4] = 2.0
    kw = dict(gamma_post=None, gate=None, gamma_pre=torch.ones(d, device="cuda"), res_scale=1.0)
    out = moe.norm_residual(r, y, eps=1e-6, **kw)
    _check_forward(out, r, y, kw)
    assert np.array_equal(to_np(out.r[:4]), np.zeros((4, d)))
    assert np.all(to_np(out.n[:4]) == 0) and np.allclose(to_np(out.rstd_pre[:4]), 1e3, rtol=1e-6)
    kw["gamma_post"] = torch.ones(d, device="cuda")
    out = moe.norm_residual(r, y, eps=1e-6, **kw)
    dr, dn = torch.ones(T, d, device="cuda"), torch.ones(T, d, device="cuda", dtype=torch.bfloat16)
    args = _backward_args(out, kw)
    _check_backward(moe.norm_residual_backward(out.r, dr, dn, y, **args), out.r, y, dr, dn, args)


def test_a_row_that_is_not_finite_stays_alone():
    """A NaN or an infinity in one token's row reaches no other row."""
    c = (40, 576, torch.float32, "both", "channel", 1.0)
    r, y, kw, _ = _case(c)
    ref = moe.norm_residual(r, y, **kw)
    r2, y2 = r.clone(), y.clone()
    r2[7, 5] = float("nan")
    y2[11, 570] = float("inf")
    out = moe.norm_residual(r2, y2, **kw)
    keep = torch.tensor([t for t in range(40) if t not in (7, 11)], device="cuda")
    for k in ("r", "n", "rstd_post", "rstd_pre"):
        assert torch.equal(getattr(out, k)[keep], getattr(ref, k)[keep])
    assert bool(torch.isnan(out.n[7]).all()) and bool(torch.isnan(out.r[11, 570]))


def test_offsets_past_32_bits():
    """Rows that begin beyond 2^31 elements."""
    T, d = (1 << 31) // 8192 + 37, 8192
    g = torch.Generator(device="cuda").manual_seed(5)
    r = torch.zeros((T, d), dtype=torch.bfloat16, device="cuda")
    y = torch.zeros((T, d), dtype=torch.bfloat16, device="cuda")
    r[-40:] = torch.randn(40, d, generator=g, device="cuda").to(torch.bfloat16)
    y[-40:] = torch.randn(40, d, generator=g, device="cuda").to(torch.bfloat16)
    kw = dict(gamma_post=torch.rand(d, generator=g, device="cuda"), gate=None,
              gamma_pre=torch.rand(d, generator=g, device="cuda"), res_scale=1.0)
    out = moe.norm_residual(r, y, **kw)
    last = moe.NormResidual(out.r[-40:], out.n[-40:], out.rstd_post[-40:], out.rstd_pre[-40:])
    _check_forward(last, r[-40:], y[-40:], kw)
    dn = torch.zeros((T, d), dtype=torch.bfloat16, device="cuda")
    dn[-40:] = torch.randn(40, d, generator=g, device="cuda").to(torch.bfloat16)
    got = moe.norm_residual_backward(out.r, r, dn, y, **_backward_args(out, kw))
    ref = op.norm_residual_backward(to_np(last.r), to_np(r[-40:]), to_np(dn[-40:]), to_np(y[-40:]),
                                    **_np(_backward_args(last, kw)))
    C = _c(d) * ULP
    for t, (value, mag), c in ((got.dr[-40:], ref["dr"], 2 * C), (got.dy[-40:], ref["dy"], 4 * C)):
        check_within(t, value, c * mag)
    # the rows before the last 40 hold zeros, so the sums over the tokens are those of the last 40
    for k, c in (("dgamma_pre", 2 * C), ("dgamma_post", 4 * C)):
        value, mag = ref[k]
        assert np.all(np.abs(to_np(getattr(got, k)) - value) <= (c + 40 * ULP) * mag)


def test_package_refusals():
    r = torch.zeros(4, 64, device="cuda")
    g = torch.ones(64, device="cuda")
    y = torch.zeros(4, 64, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="contiguous"):
        moe.norm_residual(torch.zeros(4, 128, device="cuda")[:, :64], gamma_pre=g)
    with pytest.raises(ValueError, match="gate"):
        moe.norm_residual(r, y, gate=torch.ones(4, 2, device="cuda"))
    with pytest.raises(TypeError, match="y must be"):
        moe.norm_residual(r, r)
    with pytest.raises(moe.MoEError):
        moe.norm_residual(r, gamma_pre=g, res_scale=0.5)
    with pytest.raises(moe.MoEError):
        moe.norm_residual(r, y, gamma_pre=g, eps=0.0)
    with pytest.raises(ValueError, match="rstd_pre"):
        moe.norm_residual_backward(r, r, y, gamma_pre=g)
