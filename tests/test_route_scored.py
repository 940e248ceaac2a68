"""GPU parity of routing by scores against oracle/operators.py (fp64).

Bounds.  A sigmoid score takes exp (2 ulp), an addition and a division: under
4 ulp of itself.  A softmax score takes l - max (rounded: 0.5 ulp of the
difference D, a relative error of D ulp after exp), exp, eight rounded
additions of positive terms and a division: under (12 + 2 D) ulp.  Adding the
bias, and two scores of a run, round once each: c is within (12 + 2 D) 2^-24 s
+ 2^-24 |c|, a run's score within its two of those and a rounding.  Each choice
must be one that values within these errors give (op.valid_choice), and where
fp64 gives it for every such value, that one.  Weights: the K-term sum and two
more roundings on top, (24 + K + 2 D) 2^-24 relative.  The gradients take about
twice as many steps: (64 + 8 D) 2^-24 of the sum of their terms' magnitudes.
Counts, offsets and the dispatch order are exact given the choice."""
import numpy as np
import pytest
import torch

import dropless_moe_expert_gb300 as moe
import oracle
from oracle import operators as op

from _helpers import to_np

pytestmark = pytest.mark.gpu
ULP = 2.0 ** -24

# T, E, K, score, n_group, topk_group, group_top, renorm, scale, bias
CASES = [
    (1, 256, 8, "sigmoid", 8, 4, 2, True, 2.5, True),
    (16, 256, 8, "sigmoid", 8, 4, 2, True, 2.5, True),       # the most tokens of one CTA, and one more
    (17, 48, 5, "softmax", 4, 3, 2, True, 1.0, True),
    (15, 31, 16, "sigmoid", 1, 1, 1, False, 1.0, False),
    (64, 256, 8, "sigmoid", 8, 4, 2, True, 2.5, True),
    (200, 192, 7, "softmax", 6, 3, 1, True, 1.0, True),      # runs of 32, one or two of their experts
    (77, 192, 7, "sigmoid", 6, 2, 2, False, 1.0, False),
    (90, 128, 4, "sigmoid", 4, 1, 2, True, 1.0, True),
    (65, 256, 8, "softmax", 8, 3, 1, False, 16.0, False),
    (1000, 256, 8, "sigmoid", 8, 4, 2, True, 2.5, True),
    (4097, 64, 6, "softmax", 1, 1, 1, False, 1.0, True),
    (2500, 128, 8, "softmax", 1, 1, 1, True, 1.0, False),
    (333, 160, 6, "softmax", 8, 3, 1, False, 16.0, False),
    (300, 60, 4, "softmax", 1, 1, 1, False, 1.0, False),
    (129, 37, 5, "sigmoid", 1, 1, 1, False, 1.0, True),
    (77, 63, 7, "sigmoid", 3, 2, 2, True, 1.0, True),
    (200, 256, 16, "sigmoid", 16, 1, 2, True, 1.0, True),    # K fills the only open run
    (200, 256, 16, "sigmoid", 256, 16, 2, True, 1.0, True),  # runs of one expert
    (50, 256, 12, "softmax", 64, 3, 2, True, 1.0, False),    # runs of four
    (90, 8, 8, "sigmoid", 2, 2, 2, True, 1.0, True),         # every expert chosen
    (40, 1, 1, "softmax", 1, 1, 1, True, 1.0, False),
    (127, 33, 16, "sigmoid", 1, 1, 1, True, -0.5, True),
    (63, 96, 3, "sigmoid", 2, 1, 1, True, 1.0, False),
    (129, 192, 10, "softmax", 12, 5, 2, True, 1.0, True),
    (8192, 64, 6, "softmax", 1, 1, 1, False, 1.0, True),     # the fewest tokens of the kernel for many
    (8203, 256, 8, "sigmoid", 8, 4, 2, True, 2.5, True),
    (8239, 100, 12, "sigmoid", 1, 1, 1, True, 1.0, False),
    (8201, 160, 16, "softmax", 8, 3, 1, True, 1.0, True),
    (8255, 20, 3, "softmax", 5, 2, 2, True, -0.5, True),
    (8192, 63, 5, "sigmoid", 3, 2, 2, True, 1.0, True),      # not in fours
]


def _case(c, seed=0):
    T, E, K, score, ng, tg, gt, renorm, scale, bias = c
    g = np.random.default_rng(seed)
    L = (g.normal(size=(T, E)) * 1.5 + 0.5 * g.normal(size=E)).astype(np.float32)
    b = (0.1 * g.normal(size=E)).astype(np.float32) if bias else None
    rule = moe.RouteRule(score, ng, tg, gt, renorm, scale)
    return L, b, rule


def _dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _spread(L):
    return (L.max(axis=1) - L.min(axis=1)).astype(np.float64)[:, None]


def _check_dispatch(r, T, E, K):
    idx = to_np(r.topk_idx)
    counts, offsets = oracle.expert_counts(idx, E)
    src_tok, row_of = oracle.dispatch_order(idx, E)
    assert np.array_equal(to_np(r.counts), counts) and np.array_equal(to_np(r.offsets), offsets)
    assert np.array_equal(to_np(r.row_of), row_of) and np.array_equal(to_np(r.src_tok), src_tok)


@pytest.mark.parametrize("c", CASES, ids=str)
def test_forward(c):
    T, E, K, score, ng, tg, gt, renorm, scale, _ = c
    L, b, rule = _case(c)
    r = moe.route_scored(_dev(L), K, rule, _dev(b))
    idx, w, s = op.route_scored(L, K, score, ng, tg, gt, renorm, scale, b)
    got = to_np(r.topk_idx)
    D = _spread(L) if score == "softmax" else np.zeros((T, 1))
    c = s if b is None else s + b.astype(np.float64)
    err = (12 + 2 * D) * ULP * s + ULP * np.abs(c)
    gerr = 2 * err.reshape(T, ng, -1).max(axis=2) + ULP * np.abs(op.run_scores(c, ng, gt))
    assert op.valid_choice(got, c, err, K, ng, tg, gt, gerr).all()
    assert (got != idx).any(axis=1).sum() <= 1 + T * 8 * K * E * 32 * ULP   # about K E 32 ulp of the tokens are near ties
    ref = op.route_scored_weights(L, got, score, renorm, scale)
    assert np.all(np.abs(to_np(r.topk_w) - ref) <= (24 + K + 2 * D) * ULP * np.abs(ref))
    _check_dispatch(r, T, E, K)


@pytest.mark.parametrize("c", CASES, ids=str)
def test_backward(c):
    T, E, K, score, ng, tg, gt, renorm, scale, _ = c
    L, b, rule = _case(c, 1)
    idx, *_ = op.route_scored(L, K, score, ng, tg, gt, renorm, scale, b)
    dw = np.random.default_rng(2).normal(size=(T, K)).astype(np.float32)
    out = torch.full((T, E), float("nan"), device="cuda")
    moe.route_scored_backward(_dev(L), _dev(idx), _dev(dw), rule, out=out)
    ref, mag = op.route_scored_backward(L, idx, dw, score, renorm, scale)
    D = _spread(L) if score == "softmax" else np.zeros((T, 1))
    assert np.all(np.abs(to_np(out) - ref) <= (64 + 8 * D) * ULP * mag)


def test_one_renormalised_choice_has_no_gradient():
    """K = 1 with renorm: the weight is scale whatever the logits, so every entry is zero, not nearly zero."""
    L, dw = torch.randn(300, 64).cuda(), torch.randn(300, 1).cuda()
    for score in ("sigmoid", "softmax"):
        rule = moe.RouteRule(score, 4, 2, 2, True, 2.5)
        r = moe.route_scored(L, 1, rule)
        assert bool((r.topk_w == 2.5).all())
        assert not bool(moe.route_scored_backward(L, r.topk_idx, dw, rule).any())


def test_ties_and_signed_zeros():
    for score in ("sigmoid", "softmax"):
        for L in (torch.zeros(70, 256), -torch.zeros(70, 256)):
            L[::2, 1::2] *= -1.0   # -0.0 and +0.0 are equal
            r = moe.route_scored(L.cuda(), 8, moe.RouteRule(score, 8, 4, 2))
            assert to_np(r.topk_idx).tolist() == [list(range(8))] * 70
            assert np.allclose(to_np(r.topk_w), 0.125, rtol=1e-6)
    # runs of 32 of equal experts; one run ahead by one expert, one by two equal ones
    L = torch.zeros(5, 256)
    L[:, 96] = 1.0
    L[:, [160, 191]] = 0.75
    r = moe.route_scored(L.cuda(), 6, moe.RouteRule("sigmoid", 8, 2, 2))
    assert to_np(r.topk_idx).tolist() == [[96, 160, 191, 97, 98, 99]] * 5
    r = moe.route_scored(L.cuda(), 4, moe.RouteRule("sigmoid", 8, 3, 1))
    assert to_np(r.topk_idx).tolist() == [[96, 160, 191, 0]] * 5
    # equal runs: the lower ones stay open; equal experts inside: the lower ones
    L = torch.zeros(3, 64)
    L[:, 32:] = 1.0
    r = moe.route_scored(L.cuda(), 5, moe.RouteRule("sigmoid", 8, 2, 2))
    assert to_np(r.topk_idx).tolist() == [[32, 33, 34, 35, 36]] * 3


def test_runs_beat_their_members():
    # the largest expert sits in a run that loses by its two best
    L = torch.full((2, 32), -4.0)
    L[:, 5] = 3.0                          # run 0: one strong expert
    L[:, 8:10] = 2.0                       # run 1
    L[:, 16:18] = 1.9                      # run 2
    r = moe.route_scored(L.cuda(), 3, moe.RouteRule("sigmoid", 4, 2, 2))
    assert to_np(r.topk_idx).tolist() == [[8, 9, 16]] * 2
    r = moe.route_scored(L.cuda(), 3, moe.RouteRule("sigmoid", 4, 2, 1))
    assert to_np(r.topk_idx).tolist() == [[5, 8, 9]] * 2


def test_closed_experts():
    """A bias of -inf closes an expert: chosen only where too few others are open."""
    g = torch.Generator().manual_seed(0)
    L = torch.randn(100, 32, generator=g)
    b = torch.zeros(32)
    b[8:] = -float("inf")
    r = moe.route_scored(L.cuda(), 6, moe.RouteRule(), b.cuda())
    assert to_np(r.topk_idx).max() < 8
    r = moe.route_scored(L.cuda(), 10, moe.RouteRule(), b.cuda())
    got = to_np(r.topk_idx)
    assert np.array_equal(got[:, 8:], np.tile([8, 9], (100, 1))) and got[:, :8].max() < 8
    # every expert closed, in runs as well: the lowest indexes, with their own weights
    b[:] = -float("inf")
    r = moe.route_scored(L.cuda(), 6, moe.RouteRule("sigmoid", 4, 2, 2), b.cuda())
    assert to_np(r.topk_idx).tolist() == [[0, 1, 2, 3, 4, 5]] * 100
    ref = op.route_scored_weights(L.numpy(), to_np(r.topk_idx))
    assert np.all(np.abs(to_np(r.topk_w) - ref) <= 40 * ULP * ref)


def test_extreme_logits():
    """Scores that saturate or vanish keep finite weights; a row of vanished scores gives zeros."""
    L = torch.tensor([[200.0, 100.0, 0.0, -100.0], [-200.0, -200.0, -200.0, -200.0], [-80.0, -81.0, -82.0, -83.0]])
    for renorm in (True, False):
        r = moe.route_scored(L.cuda(), 2, moe.RouteRule(renorm=renorm))
        assert to_np(r.topk_idx).tolist() == [[0, 1], [0, 1], [0, 1]]
        w = to_np(r.topk_w)
        assert np.all(np.isfinite(w)) and np.array_equal(w[1], [0.0, 0.0])
        assert np.array_equal(w[0], [0.5, 0.5] if renorm else [1.0, 1.0])
        ref = op.route_scored_weights(L.numpy(), to_np(r.topk_idx), "sigmoid", renorm)
        assert np.all(np.abs(w[2] - ref[2]) <= 30 * ULP * ref[2])
    r = moe.route_scored(L.cuda(), 2, moe.RouteRule("softmax", renorm=False))
    assert np.all(np.abs(to_np(r.topk_w)[0] - [1.0, 0.0]) <= 1e-30)
    d = moe.route_scored_backward(L.cuda(), r.topk_idx, torch.ones(3, 2).cuda(), moe.RouteRule())
    assert np.all(np.isfinite(to_np(d)))


def test_masked_logits():
    """A logit of -inf is a score of zero; the others are as if it were not there."""
    g = torch.Generator().manual_seed(1)
    L = torch.randn(70, 64, generator=g)
    M = L.clone()
    M[:, 40:] = -float("inf")
    for score in ("sigmoid", "softmax"):
        rule = moe.RouteRule(score, renorm=False)
        a = moe.route_scored(M.cuda(), 5, rule)
        b = moe.route_scored(L[:, :40].contiguous().cuda(), 5, rule)
        assert torch.equal(a.topk_idx, b.topk_idx) and torch.equal(a.topk_w, b.topk_w)
        d = moe.route_scored_backward(M.cuda(), a.topk_idx, torch.ones(70, 5).cuda(), rule)
        assert bool(torch.isfinite(d).all()) and not bool(d[:, 40:].any())


def test_buffers_streams_and_bits():
    """The same bits on every call, on another stream, into reused buffers, and from a captured graph."""
    case = CASES[3]
    L, b, rule = _case(case)
    Ld, bd = _dev(L), _dev(b)
    T, E, K = case[:3]
    ref = moe.route_scored(Ld, K, rule, bd)
    buf = moe.RouteBuffers(T, E, K)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    first = moe.launch_count()
    with torch.cuda.stream(side):
        got = moe.route_scored(Ld, K, rule, bd, buffers=buf)
    torch.cuda.current_stream().wait_stream(side)
    assert moe.launch_count() > first and got is buf.routing
    graph = torch.cuda.CUDAGraph()
    other = moe.RouteBuffers(T, E, K)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        moe.route_scored(Ld, K, rule, bd, buffers=other)
    for t in vars(other.routing).values():
        t.fill_(-1)
    graph.replay()
    torch.cuda.synchronize()
    for name in vars(ref):
        for r in (got, other.routing):
            assert torch.equal(getattr(r, name).view(torch.int32), getattr(ref, name).view(torch.int32)), name
    with pytest.raises(ValueError, match="buffers"):
        moe.route_scored(Ld[:10], K, rule, bd, buffers=buf)


def test_offsets_past_32_bits():
    """Logits of more than 2^31 elements (the last tokens are checked)."""
    T, E, K = (1 << 23) + 77, 256, 4
    L = torch.zeros((T, E), device="cuda")
    tail = np.random.default_rng(3).normal(size=(64, E)).astype(np.float32)
    L[-64:] = _dev(tail)
    rule = moe.RouteRule(renorm=False)
    r = moe.route_scored(L, K, rule)
    idx, *_ = op.route_scored(tail, K, renorm=False)
    assert np.array_equal(to_np(r.topk_idx[-64:]), idx)
    assert r.topk_idx[:1000].cpu().tolist() == [[0, 1, 2, 3]] * 1000
    assert int(r.offsets[-1]) == T * K and int(r.counts.sum()) == T * K
    d = moe.route_scored_backward(L, r.topk_idx, torch.ones((T, K), device="cuda"), rule)
    ref, mag = op.route_scored_backward(tail, idx, np.ones((64, K)), renorm=False)
    assert np.all(np.abs(to_np(d[-64:]) - ref) <= 64 * ULP * mag)


@pytest.mark.parametrize("c", [
    (8192, 64, 6, "softmax", 1, 1, 1, True, 1.0, True), (8205, 256, 8, "sigmoid", 8, 4, 2, True, 2.5, True),
    (9000, 128, 16, "softmax", 16, 4, 2, True, 1.0, False), (8230, 36, 9, "sigmoid", 3, 2, 1, False, 1.0, True),
    (5123, 240, 7, "softmax", 1, 1, 1, False, 1.0, True), (8200, 64, 16, "sigmoid", 16, 4, 2, True, 1.0, True),
    (8192, 20, 20 - 4, "softmax", 1, 1, 1, True, 1.0, False)], ids=str)
def test_the_same_bits_among_many_tokens_as_among_few(c):
    T, E, K = c[:3]
    L, b, rule = _case(c)
    L[::7] = np.round(L[::7])                    # ties
    L[3::97] = 0.0
    L[5::101, 1::3] = -np.inf
    L[6::103, 2] = np.inf
    L[8::107, E // 2] = np.nan
    L[9::109] = -np.inf
    L[10::113, ::2] = -0.0
    L[11::127] *= 1e30
    many = moe.route_scored(_dev(L), K, rule, _dev(b))
    _check_dispatch(many, T, E, K)
    for i in range(0, T, 1024):
        few = moe.route_scored(_dev(L[i:i + 1024]), K, rule, _dev(b))
        assert torch.equal(many.topk_idx[i:i + 1024], few.topk_idx)
        assert torch.equal(many.topk_w[i:i + 1024].view(torch.int32), few.topk_w.view(torch.int32))


def test_addresses_that_are_not_on_sixteen_bytes():
    """Among many tokens too: the logits and the bias at any fp32 address."""
    T, E, K = 8192, 64, 6
    L, b, rule = _case((T, E, K, "sigmoid", 4, 2, 2, True, 1.0, True))
    ref = moe.route_scored(_dev(L), K, rule, _dev(b))
    held = torch.empty(T * E + 1, device="cuda")
    bias = torch.empty(E + 1, device="cuda")
    held[1:] = _dev(L).flatten()
    bias[1:] = _dev(b)
    for logits, add in ((held[1:].view(T, E), _dev(b)), (_dev(L), bias[1:])):
        r = moe.route_scored(logits, K, rule, add)
        assert torch.equal(r.topk_idx, ref.topk_idx)
        assert torch.equal(r.topk_w.view(torch.int32), ref.topk_w.view(torch.int32))
