"""GPU parity of the norms, gate and residual with dropout against
oracle/operators.py (fp64): the mask exactly, the rest within the bounds of
tests/test_norm_residual.py, whose roundings these kernels share (one more
for the kept elements' factor is inside the 16 that C allows)."""
import numpy as np
import pytest
import torch

import dropless_moe_expert_gb300 as moe
from oracle import operators as op

from _bounds import check_within
from _helpers import to_np

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
ULP = 2.0 ** -24

# T, d, residual, gamma_post, gamma_pre, gate, res_scale, p
CASES = [(1, 64, BF16, 0, 0, "none", 1.0, 0.5), (1, 7168, F32, 1, 1, "channel", 1.0, 0.1),
         (7, 128, BF16, 0, 1, "token", 0.5, 0.3), (129, 1024, BF16, 0, 0, "none", 1.0, 0.1),
         (300, 4096, BF16, 1, 1, "channel", 0.5, 0.1), (517, 192, F32, 1, 1, "token", 0.7, 0.25),
         (129, 2368, F32, 1, 0, "channel", 1.0, 0.05), (65, 2368, BF16, 0, 1, "none", 1.0, 0.9),
         (33, 16384, F32, 1, 1, "channel", 1.0, 0.1), (33, 16384, BF16, 1, 1, "none", 1.0, 0.1),
         (20, 8256, BF16, 1, 1, "token", 1.0, 0.2), (300, 320, BF16, 1, 1, "none", 1.0, 1 / 65536),
         (200, 7168, F32, 0, 1, "token", 1.0, 0.25), (457, 512, BF16, 1, 1, "channel", 1.0, 0.1),
         (170, 5120, BF16, 0, 1, "channel", 1.0, 0.1), (160, 5120, F32, 1, 0, "token", 1.0, 0.1),
         (310, 256, F32, 0, 0, "token", 0.0, 65535 / 65536), (155, 12288, F32, 0, 0, "token", 1.0, 0.4),
         (161, 12352, BF16, 1, 0, "channel", 1.0, 0.1), (333, 1536, F32, 1, 1, "channel", 0.5, 0.3)]
SEEDS = [(0, 0), (-1, -1), (0x0123456789abcdef, 1 << 40), (77, 3)]
WORD = (1 << 64) - 1


def _rng(k):
    return torch.tensor(SEEDS[k % 4], device="cuda")


def _mask(T, d, p, rng, rows=None):
    seed, call = (v & WORD for v in rng.tolist())
    return op.dropout_mask(T, d, p, seed, call, rows)


def _case(c, seed=0):
    T, d, dt, post, pre, gate, a, p = c
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*s):
        return torch.randn(*s, generator=g, device="cuda")

    kw = dict(gamma_post=1 + 0.2 * normal(d) if post else None, gamma_pre=1 + 0.2 * normal(d) if pre else None,
              gate={"none": None, "channel": 0.3 * normal(d), "token": normal(T, 1)}[gate], res_scale=a)
    r, y = (3.0 * normal(T, d)).to(dt), (0.3 * normal(T, d)).to(BF16)
    return r, y, kw, normal(T, d).to(dt), normal(T, d).to(BF16) if pre else None


def _np(kw):
    return {k: to_np(v) if isinstance(v, torch.Tensor) else v for k, v in kw.items()}


def _check_forward(out, r, y, kw, mask):
    x, n, rp, rq, mag = op.norm_residual(to_np(r), to_np(y), mask=mask, **_np(kw))
    C = (r.shape[1] / 8 + 32) * ULP
    check_within(out.r, x, C * mag + 1e-38, "r")
    if rp is not None:
        assert np.all(np.abs(to_np(out.rstd_post) - rp) <= 2 * C * rp)
    if n is not None:
        slack = np.sqrt(np.mean(mag ** 2, axis=1)) * rq
        assert np.all(np.abs(to_np(out.rstd_pre) - rq) <= C * rq * (1 + slack))
        row = np.sqrt(np.mean(mag ** 2, axis=1, keepdims=True))
        tol = 2 * C * rq[:, None] * np.abs(_np(kw)["gamma_pre"]) * (mag + np.abs(x) * (1 + row * rq[:, None]))
        check_within(out.n, n, tol + 1e-38, "n")


def _check_backward(got, r2, y, dr, dn, args, mask):
    ref = op.norm_residual_backward(to_np(r2), None if dr is None else to_np(dr), None if dn is None else to_np(dn),
                                    to_np(y), mask=mask, **_np(args))
    T, d = r2.shape
    C = (d / 8 + 32) * ULP
    for name, t, c in (("dr", got.dr, 2 * C), ("dy", got.dy, 4 * C), ("dgamma_pre", got.dgamma_pre, 2 * C + T * ULP),
                       ("dgamma_post", got.dgamma_post, 4 * C + T * ULP), ("dgate", got.dgate, 4 * C + T * ULP)):
        assert (t is not None) == (name in ref), name
        if t is not None:
            value, mag = ref[name]
            check_within(t, value, c * mag + 1e-37, name)


def _args(out, kw):
    return dict(kw, rstd_post=out.rstd_post, rstd_pre=out.rstd_pre)


@pytest.mark.parametrize("k", range(len(CASES)), ids=[str(c) for c in CASES])
def test_forward_and_backward(k):
    c = CASES[k]
    T, d, p = c[0], c[1], c[-1]
    r, y, kw, dr, dn = _case(c)
    rng = _rng(k)
    mask = _mask(T, d, p, rng)
    out = moe.norm_residual(r, y, dropout=p, rng=rng, **kw)
    _check_forward(out, r, y, kw, mask)
    assert torch.equal(out.rng, rng) and out.rng.data_ptr() != rng.data_ptr()
    args = _args(out, kw)
    got = moe.norm_residual_backward(out.r, dr, dn, y, dropout=p, rng=out.rng, **args)
    _check_backward(got, out.r, y, dr, dn, args, mask)
    again = moe.norm_residual_backward(out.r, dr, dn, y, dropout=p, rng=rng, **args)
    for name, v in vars(got).items():
        if v is not None and name != "workspace" and not name.startswith("_"):
            assert torch.equal(v, vars(again)[name]), name
    if dn is not None:
        got = moe.norm_residual_backward(out.r, None, dn, y, dropout=p, rng=rng, **args)
        _check_backward(got, out.r, y, None, dn, args, mask)


def test_the_mask_by_itself():
    """r' = drop(1): zeros and 1 / (1 - p), exactly the oracle's, the share within six deviations, and another
    call number another mask."""
    T, d, p = 500, 256, 0.1
    zero, one = torch.zeros(T, d, device="cuda"), torch.ones(T, d, device="cuda", dtype=BF16)
    masks = []
    for call in (0, 1):
        rng = torch.tensor([42, call], device="cuda")
        m = moe.norm_residual(zero, one, dropout=p, rng=rng).r
        ref = _mask(T, d, p, rng)
        assert np.array_equal(to_np(m), ref.astype(np.float32))
        assert abs((ref > 0).mean() - 0.9) < 6 * np.sqrt(0.09 / ref.size)
        masks.append(ref > 0)
    both = (masks[0] & masks[1]).mean()
    assert abs(both - 0.81) < 6 * np.sqrt(0.81 * 0.19 / (T * d))


def test_without_dropout_nothing_changes():
    c = CASES[4]
    r, y, kw, dr, dn = _case(c)
    a, b = moe.norm_residual(r, y, **kw), moe.norm_residual(r, y, dropout=0.0, rng=_rng(0), **kw)
    assert torch.equal(a.r, b.r) and torch.equal(a.n, b.n) and b.rng is None
    # below half a step of 2^-16 nothing is dropped either
    t = moe.norm_residual(r, y, dropout=2.0 ** -19, rng=_rng(0), **kw)
    _check_forward(t, r, y, kw, np.ones((c[0], c[1])))


@pytest.mark.parametrize("post", [0, 1])
def test_dropped_elements_are_left_out_whatever_they_are(post):
    """A NaN or an infinity that is dropped reaches nothing (with a norm before it: nothing of its row's dropped places)."""
    c = (40, 576, F32, post, 1, "channel", 1.0, 0.5)
    r, y, kw, dr, dn = _case(c)
    rng = _rng(3)
    mask = _mask(40, 576, 0.5, rng)
    dropped = np.argwhere(mask[7] == 0)[:2, 0]
    y2 = y.clone()
    y2[7, int(dropped[0])], y2[7, int(dropped[1])] = float("nan"), float("inf")
    out, ref = (moe.norm_residual(r, t, dropout=0.5, rng=rng, **kw) for t in (y2, y))
    gone = torch.from_numpy(mask == 0).cuda()
    assert torch.equal(out.r[gone], ref.r[gone])
    if not post:
        assert torch.equal(out.r, ref.r) and torch.equal(out.n, ref.n)
        a, b = (moe.norm_residual_backward(ref.r, dr, dn, t, dropout=0.5, rng=rng, **_args(ref, kw)) for t in (y2, y))
        for k in ("dr", "dy", "dgamma_pre", "dgate"):
            assert torch.equal(getattr(a, k), getattr(b, k)), k


def test_buffers_streams_and_graphs():
    """In place, reused buffers, another stream; a captured step draws anew from a call number that the graph
    itself counts up, and its backward draws the same."""
    c = (203, 1088, BF16, 1, 1, "channel", 0.5, 0.2)
    T, d, p = c[0], c[1], c[-1]
    r, y, kw, dr, dn = _case(c)
    rng = torch.tensor([123, 7], device="cuda")
    ref = moe.norm_residual(r, y, dropout=p, rng=rng, **kw)
    gref = moe.norm_residual_backward(ref.r, dr, dn, y, dropout=p, rng=ref.rng, **_args(ref, kw))
    out = moe.NormResidual.empty(T, d, BF16, rng=True)
    out.r = r.clone()
    gout = moe.NormResidualGrads.empty(T, d, BF16, gate="channel")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        moe.norm_residual(out.r, y, dropout=p, rng=rng, out=out, **kw)
        moe.norm_residual_backward(out.r, dr, dn, y, dropout=p, rng=out.rng, out=gout, **_args(out, kw))
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out.r, ref.r) and torch.equal(gout.dy, gref.dy) and torch.equal(gout.dgate, gref.dgate)
    given = moe.norm_residual(r, y, dropout=p, rng=rng, stream=side, **kw)
    torch.cuda.synchronize()
    assert torch.equal(given.r, ref.r) and torch.equal(given.rng, rng)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a = moe.norm_residual(r, y, dropout=p, rng=rng, **kw)
        rng[1] += 1
        g = moe.norm_residual_backward(a.r, dr, dn, y, dropout=p, rng=a.rng, **_args(a, kw))
    for call in (7, 8, 9):
        graph.replay()
        torch.cuda.synchronize()
        assert a.rng.tolist() == [123, call]
        mask = _mask(T, d, p, a.rng)
        _check_forward(a, r, y, kw, mask)
        _check_backward(g, a.r, y, dr, dn, _args(a, kw), mask)


def test_offsets_past_32_bits():
    """Rows that begin beyond element 2^32."""
    T, d, p, n = (1 << 32) // 8192 + 21, 8192, 0.25, 6
    r = torch.zeros((T, d), dtype=BF16, device="cuda")
    y = torch.zeros((T, d), dtype=BF16, device="cuda")
    y[-n:] = 1.0
    rng = _rng(2)
    out = moe.norm_residual(r, y, dropout=p, rng=rng, out=None)
    mask = _mask(T, d, p, rng, rows=range(T - n, T))
    assert np.array_equal(to_np(out.r[-n:]), to_np(torch.from_numpy(mask).to(BF16)))
    got = moe.norm_residual_backward(out.r, y, None, y, dropout=p, rng=rng)
    assert np.array_equal(to_np(got.dy[-n:]), to_np(torch.from_numpy(mask).to(BF16)))


def test_refusals():
    r, y = torch.zeros(4, 64, device="cuda"), torch.zeros(4, 64, device="cuda", dtype=BF16)
    rng, g = _rng(0), torch.ones(64, device="cuda")
    with pytest.raises(ValueError, match="rng"):
        moe.norm_residual(r, y, dropout=0.1)
    with pytest.raises(TypeError, match="rng"):
        moe.norm_residual(r, y, dropout=0.1, rng=rng.int())
    with pytest.raises(ValueError, match="CUDA"):
        moe.norm_residual(r, y, dropout=0.1, rng=rng.cpu())
    for p in (-0.1, 1.0, 1.5, float("nan"), 1 - 2.0 ** -18):
        with pytest.raises(moe.MoEError, match="INVALID"):
            moe.norm_residual(r, y, dropout=p, rng=rng)
        with pytest.raises(moe.MoEError, match="INVALID"):
            moe.norm_residual_backward(r, r, None, y, dropout=p, rng=rng)
    with pytest.raises(moe.MoEError, match="INVALID"):      # nothing that it acts on
        moe.norm_residual(r, gamma_pre=g, dropout=0.1, rng=rng)
    assert moe.device_status() == 0
