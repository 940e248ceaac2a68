"""GPU parity of the gated feed-forward and its gradients against
oracle/operators.py (fp64).

Bounds, element by element, from the roundings on the way.
- A sum of K products: the tensor cores add 16 at a time to an fp32 value, so
  the error is under (K / 16 + 16) steps of 2^-23 of the sum of the terms'
  magnitudes S (a step of truncation each; a split of K adds fewer than 8 more).
- An activation of g: exp(z) by ex2 is within (2 + 1.2 |z|) 2^-23, z itself within
  2^-22 |z|, the rest a few roundings: together (8 + 4 |z|) 2^-23 of the terms'
  magnitudes, with z as in the code, or g^2 / 2 for the normal density.
- h and da are rounded to bf16 once: 2^-8 of their values, and carry through
  the next product by the magnitudes of its other factor.  An output's own
  rounding is exact in _bounds.within.
Over a whole output the two roundings of a value that passes h are
independent, each at most 2^-8 relative and 2^-8 / sqrt(3) in the mean square:
relative L2 under 2^-8."""
import numpy as np
import pytest
import torch

import dropless_moe_expert_gb300 as moe
from oracle import operators as op

from _bounds import check_within
from _helpers import rel_l2, to_np

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
HALF = 2.0 ** -8
STEP = 2.0 ** -23
ACTS = ("silu", "gelu", "gelu_tanh", "relu")

# T, d, f, act: few tokens (blocks of 16 to 128, with and without a split of K), tiles of CTA pairs, sizes that fill nothing
CASES = [(1, 8, 8, "silu"), (1, 64, 128, "gelu"), (2, 2056, 264, "silu"), (1, 7168, 2048, "silu"), (5, 96, 472, "gelu_tanh"),
         (16, 1024, 136, "relu"), (17, 136, 1032, "silu"), (37, 2048, 768, "gelu_tanh"), (64, 512, 4096, "gelu"),
         (100, 1416, 520, "silu"), (128, 256, 256, "relu"), (129, 328, 776, "silu"), (200, 128, 128, "gelu"),
         (257, 8, 16, "silu"), (300, 1032, 2056, "gelu_tanh"), (600, 4096, 24, "silu"), (777, 200, 1000, "gelu"),
         (1003, 2056, 1368, "gelu"), (1500, 640, 1280, "relu"), (2049, 384, 640, "silu"), (4096, 1024, 2048, "gelu_tanh")]


def _case(c, seed=0):
    T, d, f, act = c
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*s):
        return torch.randn(*s, generator=g, device="cuda")

    x = normal(T, d).to(BF16)
    W1, W2 = (normal(2 * f, d) / d ** 0.5).to(BF16), (normal(d, f) / f ** 0.5).to(BF16)
    return x, W1, W2, normal(T, d).to(BF16), normal(T, d).to(BF16)     # dy, add


def _sum(K):
    return (K / 16 + 16) * STEP


def _mm(a, b):
    """A product in fp64, on the GPU where it is large."""
    return to_np(torch.from_numpy(np.ascontiguousarray(a)).cuda().double() @
                 torch.from_numpy(np.ascontiguousarray(b)).cuda().double())


def _terms(act, g):
    """act(g), act'(g), and bounds of their errors."""
    v, slope = op.activation(act, g)
    z = {"silu": np.abs(g), "gelu": 0.5 * g * g, "relu": 0 * g,
         "gelu_tanh": np.abs(1.6 * g * (1 + 0.045 * g * g))}[act]
    dz = {"silu": 1.0, "gelu": 0.4, "relu": 0.0, "gelu_tanh": 1.6 * (1 + 0.14 * g * g)}[act]
    rel = (8 + 4 * z) * STEP
    s = np.where(g == 0, 0.5, v / np.where(g == 0, 1, g))
    return v, slope, rel * np.abs(v), 2 * rel * (np.abs(s) + np.abs(g) * dz * (np.exp(-z) if act == "gelu" else np.abs(s)))


def _forward_reference(c, x, W1, W2, add=None):
    """y and a in fp64 with the bounds of their errors before the last rounding."""
    T, d, f, act = c
    x, W1, W2 = (to_np(t).astype(np.float64) for t in (x, W1, W2))
    a = _mm(x, W1.T)
    ea = _sum(d) * _mm(np.abs(x), np.abs(W1).T)
    g, u = a[:, :f], a[:, f:]
    v, _, ev, _ = _terms(act, g)
    ev = ev + 1.2 * ea[:, :f]                   # no activation is steeper than 1.2
    h = v * u
    eh = ev * np.abs(u) + (np.abs(v) + ev) * ea[:, f:]
    eh = eh + HALF * (np.abs(h) + eh)
    y = _mm(h, W2.T)
    ey = _mm(eh + _sum(f) * (np.abs(h) + eh), np.abs(W2).T)
    if add is not None:
        add = to_np(add).astype(np.float64)
        y, ey = y + add, ey + STEP * (np.abs(y) + np.abs(add))
    return y, ey + 1e-30, a, ea + 1e-30


def _check_forward(c, y, ref, pre=None):
    want, ey, a, ea = ref
    check_within(y, want, ey, "y")
    if want.size >= 4096:
        assert rel_l2(to_np(y), want) <= HALF
    if pre is not None:
        check_within(pre, a, ea, "preact")


@pytest.mark.parametrize("c", CASES, ids=str)
def test_forward(c):
    x, W1, W2, _, add = _case(c)
    T, d, f, act = c
    ref = _forward_reference(c, x, W1, W2)
    y = moe.gated_ffn(x, W1, W2, act)
    _check_forward(c, y, ref)
    pre = torch.full((T, 2 * f), float("nan"), dtype=BF16, device="cuda")
    assert torch.equal(moe.gated_ffn(x, W1, W2, act, preact=pre), y)
    _check_forward(c, y, ref, pre)
    # onto another output, apart and in place
    z = moe.gated_ffn(x, W1, W2, act, add=add)
    _check_forward(c, z, _forward_reference(c, x, W1, W2, add))
    w = add.clone()
    assert moe.gated_ffn(x, W1, W2, act, add=w, out=w) is w and torch.equal(w, z)
    assert moe.device_status() == 0


@pytest.mark.parametrize("c", [c for c in CASES if c[0] > 1] + [(1, 64, 128, "silu")], ids=str)
def test_backward(c):
    T, d, f, act = c
    x, W1, W2, dy, add = _case(c, 1)
    pre = torch.empty(T, 2 * f, dtype=BF16, device="cuda")
    moe.gated_ffn(x, W1, W2, act, preact=pre)
    out = moe.GatedFFNGrads.empty(T, d, f)
    for t in (out.dx, out.dW1, out.dW2):
        t.fill_(float("nan"))
    got = moe.gated_ffn_backward(x, pre, dy, W1, W2, act, out=out)
    assert got is out

    xs, a, ds, A, B = (to_np(t).astype(np.float64) for t in (x, pre, dy, W1, W2))
    g, u = a[:, :f], a[:, f:]
    v, slope, ev, es = _terms(act, g)
    dh, edh = _mm(ds, B), _sum(d) * _mm(np.abs(ds), np.abs(B))
    da = np.concatenate([dh * u * slope, dh * v], axis=1)
    eda = np.concatenate([np.abs(u) * (edh * np.abs(slope) + (np.abs(dh) + edh) * es),
                          edh * np.abs(v) + (np.abs(dh) + edh) * ev], axis=1)
    eda = eda + (HALF + 4 * STEP) * (np.abs(da) + eda)
    h = v * u
    eh = ev * np.abs(u)
    eh = eh + (HALF + 2 * STEP) * (np.abs(h) + eh)
    want = dict(dx=(_mm(da, A), _mm(eda + _sum(2 * f) * (np.abs(da) + eda), np.abs(A))),
                dW1=(_mm(da.T, xs), _mm((eda + _sum(T) * (np.abs(da) + eda)).T, np.abs(xs))),
                dW2=(_mm(ds.T, h), _mm(np.abs(ds).T, eh + _sum(T) * (np.abs(h) + eh))))
    for name, (value, err) in want.items():
        check_within(getattr(got, name), value, err + 1e-30, name)
        if value.size >= 4096 and T > 1:
            assert rel_l2(to_np(getattr(got, name)), value) <= HALF, name
    # the weights' gradients in fp32; alone; dx onto another one, in place
    wide = moe.gated_ffn_backward(x, pre, dy, W1, W2, act, out=moe.GatedFFNGrads.empty(T, d, f, F32, dx=False))
    assert wide.dx is None
    for name in ("dW1", "dW2"):
        check_within(getattr(wide, name), want[name][0], want[name][1] + 1e-30, name)
        assert torch.equal(getattr(wide, name).to(BF16), getattr(got, name))
    dx = add.clone()
    one = moe.gated_ffn_backward(x, pre, dy, W1, W2, act, add=dx, out=moe.GatedFFNGrads(dx))
    assert one.dW1 is None
    value, err = want["dx"]
    s = to_np(add).astype(np.float64)
    check_within(dx, value + s, err + STEP * (np.abs(value) + np.abs(s)) + 1e-30, "dx + add")
    assert moe.device_status() == 0


# what the sizes choose between: da and h, and dx, each with K shared or in large tiles
FEW = [(2, 64, 4096, "gelu"), (17, 1032, 520, "relu"), (100, 256, 2048, "silu"), (130, 96, 3000, "gelu_tanh"),
       (300, 264, 2504, "silu"), (333, 2000, 96, "gelu"), (777, 256, 4096, "silu"), (1030, 1032, 520, "gelu")]


@pytest.mark.parametrize("c", FEW, ids=str)
def test_backward_of_few_tokens_or_columns(c):
    test_backward(c)


@pytest.mark.parametrize("c", [FEW[1], FEW[3], FEW[5], FEW[6]], ids=str)
def test_few_tokens_or_columns_around_and_behind_other_work(c):
    test_what_lies_around_the_outputs_stays(c)
    test_inputs_written_just_before(c)
    test_streams_graphs_and_repeated_calls(c)


@pytest.mark.parametrize("wanted", ["dx", "dW1", "dW2", "dx dW1", "dx dW2", "dW1 dW2"])
@pytest.mark.parametrize("c", [FEW[2], FEW[6]], ids=str)
def test_only_some_of_the_gradients_of_few_tokens(c, wanted):
    """Each within the roundings of the one beside all three: dx may be summed in another order."""
    T, d, f, act = c
    x, W1, W2, dy, _ = _case(c, 1)
    pre = torch.empty(T, 2 * f, dtype=BF16, device="cuda")
    moe.gated_ffn(x, W1, W2, act, preact=pre)
    full = moe.gated_ffn_backward(x, pre, dy, W1, W2, act)
    empty = moe.GatedFFNGrads.empty(T, d, f)
    some = moe.GatedFFNGrads(*(getattr(empty, n) if n in wanted.split() else None for n in ("dx", "dW1", "dW2")))
    moe.gated_ffn_backward(x, pre, dy, W1, W2, act, out=some)
    for n in wanted.split():
        a, b = getattr(some, n), getattr(full, n)
        assert torch.equal(a, b) if n != "dx" else rel_l2(to_np(a), to_np(b).astype(np.float64)) <= HALF, n


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T", [3, 700])
def test_large_and_special_pre_activations(act, T):
    """Gates from the smallest to the largest magnitudes: through the identity as
    W1, one value per column.  A quotient by 2^126 or more is 0 in the kernels, so
    a logistic function below 2^-126 is, and |g| 2^-126 is allowed beside the bounds."""
    vals = [0.0, -0.0, 1e-30, -1e-30, 5.5, -5.5, 9.0, -9.0, 20.0, -20.0, 88.0, -88.0, 104.0, -104.0, 1e4, -1e4, 1e18, -1e18,
            1e20, -1e20, 3e38, -3e38, 0.75, -0.75, 2.5, -2.5, 13.5, -13.5, 40.0, -40.0, 3.0, -3.0]
    f = d = len(vals)
    x = torch.tensor(vals, device="cuda").to(BF16).repeat(T, 1)
    W1 = torch.cat([torch.eye(f, d), torch.zeros(f, d)]).to(BF16).cuda()
    W1[f:, 0] = 0.0
    # u = 1: from one more input that is 1
    x = torch.cat([x, torch.ones(T, 8, device="cuda", dtype=BF16)], dim=1)
    W1 = torch.cat([W1, torch.zeros(2 * f, 8, device="cuda", dtype=BF16)], dim=1)
    W1[f:, d] = 1.0
    W2 = torch.zeros(d + 8, f, device="cuda", dtype=BF16)
    W2[:d] = torch.eye(f, device="cuda").to(BF16)
    pre = torch.empty(T, 2 * f, dtype=BF16, device="cuda")
    y = moe.gated_ffn(x, W1, W2, act, preact=pre)
    g = to_np(x[0, :d]).astype(np.float64)
    assert np.array_equal(to_np(pre[T - 1, :f]), g) and bool((pre[:, f:] == 1).all())
    floor = (1 + np.minimum(np.abs(g), 200)) * 2.0 ** -125
    with np.errstate(over="ignore"):
        v, slope, ev, es = _terms(act, np.clip(g, -1e6, 1e6))
        v = np.where(np.abs(g) > 1e6, np.maximum(g, 0.0), v)
        check_within(y[:, :d], np.broadcast_to(v, (T, d)), np.minimum(ev, 1e-3 * np.abs(v)) + HALF * np.abs(v) + floor, "y")
    dy = torch.ones_like(x)
    got = moe.gated_ffn_backward(x, pre, dy, W1, W2, act)
    assert bool(torch.isfinite(got.dx).all())
    want = np.where(np.abs(g) > 1e6, (g > 0).astype(np.float64), slope)
    err = np.where(np.abs(g) > 100, 1e-6, es)
    check_within(got.dx[:, :d], np.broadcast_to(want, (T, d)), err + HALF * np.abs(want) + floor, "dx")


@pytest.mark.parametrize("c", [(3, 200, 136, "silu"), (300, 200, 136, "gelu"), (700, 512, 640, "silu")], ids=str)
def test_a_row_that_is_not_finite_stays_alone(c):
    T, d, f, act = c
    x, W1, W2, dy, _ = _case(c)
    pre, pre2 = (torch.empty(T, 2 * f, dtype=BF16, device="cuda") for _ in range(2))
    y = moe.gated_ffn(x, W1, W2, act, preact=pre)
    dx = moe.gated_ffn_backward(x, pre, dy, W1, W2, act).dx
    x2 = x.clone()
    x2[1, 5] = float("nan")
    x2[T - 1, 0] = float("inf")
    y2 = moe.gated_ffn(x2, W1, W2, act, preact=pre2)
    keep = torch.tensor([t for t in range(T) if t not in (1, T - 1)], device="cuda")
    assert torch.equal(y2[keep], y[keep]) and bool(torch.isnan(y2[1]).all()) and not bool(torch.isfinite(y2[T - 1]).any())
    assert torch.equal(moe.gated_ffn_backward(x2, pre2, dy, W1, W2, act).dx[keep], dx[keep])


@pytest.mark.parametrize("c", [(1, 256, 264, "silu"), (40, 1032, 520, "gelu"), (500, 264, 1288, "silu")], ids=str)
def test_what_lies_around_the_outputs_stays(c):
    """Outputs in the middle of larger buffers, rows behind the last token among them."""
    T, d, f, act = c
    x, W1, W2, dy, _ = _case(c)

    def inside(rows, cols, dt=BF16):
        big = torch.full((rows + 64, cols), 7.0, dtype=dt, device="cuda")
        return big, big[32:32 + rows]

    by, y = inside(T, d)
    bp, pre = inside(T, 2 * f)
    moe.gated_ffn(x, W1, W2, act, out=y, preact=pre)
    bx, dx = inside(T, d)
    b1, dW1 = inside(2 * f, d)
    b2, dW2 = inside(d, f, BF16)
    moe.gated_ffn_backward(x, pre, dy, W1, W2, act, out=moe.GatedFFNGrads(dx, dW1, dW2))
    b3, w1 = inside(2 * f, d, F32)
    b4, w2 = inside(d, f, F32)
    moe.gated_ffn_backward(x, pre, dy, W1, W2, act, out=moe.GatedFFNGrads(None, w1, w2))
    for big in (by, bp, bx, b1, b2, b3, b4):
        assert bool((big[:32] == 7).all()) and bool((big[-32:] == 7).all())
    assert torch.equal(y, moe.gated_ffn(x, W1, W2, act))


@pytest.mark.parametrize("c", [(1, 1024, 512, "silu"), (50, 512, 2048, "gelu"), (1200, 512, 776, "silu")], ids=str)
def test_streams_graphs_and_repeated_calls(c):
    """The same bits on every call, on another stream, from two captured graphs
    of one workspace replayed in turn, and with new inputs in a replay."""
    T, d, f, act = c
    x, W1, W2, dy, _ = _case(c)
    x2, dy2 = _case(c, 5)[0], _case(c, 5)[3]

    def step(a, b, ffn):
        y = ffn(a, save_preact=True)
        g = ffn.backward(a, b)
        return y, g["dx"], g["dW1"], g["dW2"]

    ffn = moe.GatedFFN(W1, W2, act, T_max=T)
    want, want2 = [t.clone() for t in step(x, dy, ffn)], [t.clone() for t in step(x2, dy2, ffn)]
    for a, b in zip(step(x, dy, ffn), want):
        assert torch.equal(a, b)
    other = moe.GatedFFN(W1, W2, act, T_max=T)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    # two calls at once, each with a workspace of its own
    with torch.cuda.stream(side):
        got = step(x, dy, other)
    again = step(x2, dy2, ffn)
    torch.cuda.current_stream().wait_stream(side)
    given = moe.gated_ffn(x, W1, W2, act, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(given, want[0])
    for a, b, e, h in zip(got, want, again, want2):
        assert torch.equal(a, b) and torch.equal(e, h)
    xs, ds = x.clone(), dy.clone()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = step(xs, ds, ffn)
        graphs.append((g, outs))
    for k, (a, b, ref) in enumerate(((x2, dy2, want2), (x, dy, want), (x2, dy2, want2))):
        xs.copy_(a)
        ds.copy_(b)
        g, outs = graphs[k % 2]
        g.replay()
        for got, r in zip(outs, ref):
            assert torch.equal(got, r)
    assert moe.device_status() == 0


@pytest.mark.parametrize("c", [(1, 1024, 2048, "silu"), (40, 2048, 768, "gelu"), (100, 4096, 1024, "silu"),
                               (300, 1024, 2048, "relu"), (1500, 1024, 1024, "silu")], ids=str)
def test_inputs_written_just_before(c):
    """Weights, tokens and the kept pre-activations change in the stream right before each call, whose kernels start
    before the ones in front of them have ended; eagerly, and in a captured graph that holds the changes too."""
    T, d, f, act = c
    sets = [_case(c, k) for k in range(3)]
    want = []
    for x, W1, W2, dy, _ in sets:
        pre = torch.empty(T, 2 * f, dtype=BF16, device="cuda")
        y = moe.gated_ffn(x, W1, W2, act, preact=pre)
        g = moe.gated_ffn_backward(x, pre, dy, W1, W2, act)
        torch.cuda.synchronize()
        want.append((y, g.dx, g.dW1, g.dW2))
    x, W1, W2, dy = (t.clone() for t in sets[2][:4])
    ffn = moe.GatedFFN(W1, W2, act, T_max=T)
    grads = moe.GatedFFNGrads.empty(T, d, f)

    def step(k):
        for to, of in ((x, 0), (W1, 1), (dy, 3), (W2, 2)):
            to.copy_(sets[k][of])
        y = ffn(x, save_preact=True)
        moe.gated_ffn_backward(x, ffn.preact, dy, W1, W2, act, out=grads)
        return [t.clone() for t in (y, grads.dx, grads.dW1, grads.dW2)]

    got = [step(k % 3) for k in range(12)]
    torch.cuda.synchronize()
    for k, outs in enumerate(got):
        for a, b in zip(outs, want[k % 3]):
            assert torch.equal(a, b), k
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [step(k) for k in (1, 0, 2, 0)]
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for k, outs in zip((1, 0, 2, 0), got):
        for a, b in zip(outs, want[k]):
            assert torch.equal(a, b), k
    assert moe.device_status() == 0


@pytest.mark.parametrize("T", [1, 48, 700])
def test_forks_and_joins_in_a_graph(T):
    """A captured graph in which the operators' kernels follow a fork, a join, a copy and one another."""
    c = (T, 512, 1024, "silu")
    x, W1, W2, dy, _ = _case(c)
    V1, V2 = _case(c, 7)[1:3]
    a, b = moe.GatedFFN(W1, W2, T_max=T), moe.GatedFFN(V1, V2, T_max=T)
    last = moe.GatedFFN(W1, W2, T_max=T)
    gamma = 1 + 0.1 * torch.randn(512, device="cuda")
    rng = torch.tensor([4, 2], device="cuda")
    xs, side = x.clone(), torch.cuda.Stream()

    def step():
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            v = b(xs, save_preact=True)
            gv = b.backward(xs, dy)
        u = a(xs, save_preact=True)
        main.wait_stream(side)
        n = moe.norm_residual(u, v, gamma_pre=gamma, dropout=0.2, rng=rng)
        y = last(n.n, save_preact=True)
        g = last.backward(n.n, dy)
        h = moe.norm_residual_backward(n.r, None, g["dx"], v, gamma_pre=gamma, rstd_pre=n.rstd_pre, dropout=0.2, rng=n.rng)
        return [u, v, n.r, y, g["dx"], g["dW1"], h.dr, h.dy, h.dgamma_pre, gv["dx"]]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    xs.copy_(dy)
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in got]
    for s, t in zip(step(), got):
        assert torch.equal(s, t)
    assert moe.device_status() == 0


def test_offsets_past_32_bits():
    """Pre-activations and their gradients that begin beyond 2^31 elements."""
    T, d, f = 70001, 8, 16384
    x, W1, W2, dy, _ = _case((T, d, f, "silu"))
    pre = torch.empty(T, 2 * f, dtype=BF16, device="cuda")
    y = moe.gated_ffn(x, W1, W2, "silu", preact=pre)
    n = 70
    c = (n, d, f, "silu")
    _check_forward(c, y[-n:], _forward_reference(c, x[-n:], W1, W2), pre[-n:])
    got = moe.gated_ffn_backward(x, pre, dy, W1, W2, "silu", out=moe.GatedFFNGrads.empty(T, d, f, weights=False))
    dx, _, _ = op.gated_ffn_backward(*(to_np(t) for t in (x[-n:], pre[-n:], dy[-n:], W1, W2)), "silu")
    assert rel_l2(to_np(got.dx[-n:]), dx) <= HALF


def test_objects():
    """What a GatedFFN keeps, and what it refuses."""
    c = (40, 128, 64, "gelu")
    x, W1, W2, dy, add = _case(c)
    ffn = moe.GatedFFN(W1, W2, "gelu", T_max=64)
    y = ffn(x)
    with pytest.raises(RuntimeError, match="save_preact"):
        ffn.backward(x, dy)
    assert torch.equal(ffn(x, save_preact=True), y)
    g = ffn.backward(x, dy, add=add)
    assert g["dW1"].dtype is F32 and g["dx"].dtype is BF16
    with pytest.raises(RuntimeError, match="tokens"):
        ffn.backward(x[:39], dy[:39])
    h = ffn.backward(x, dy, grads=dict(dW2=torch.empty_like(W2)))
    assert torch.equal(h["dW2"], g["dW2"].to(BF16))
    with pytest.raises(ValueError, match="workspace"):
        ffn(torch.zeros(65, 128, device="cuda", dtype=BF16))
    with pytest.raises(ValueError, match="act"):
        moe.GatedFFN(W1, W2, "tanh")
    with pytest.raises(ValueError, match="contiguous"):
        moe.gated_ffn(torch.zeros(4, 256, device="cuda", dtype=BF16)[:, :128], W1, W2)
    with pytest.raises(ValueError, match="W1"):
        moe.gated_ffn(x, W1[:100], W2)
    with pytest.raises(TypeError, match="x must"):
        moe.gated_ffn(x.float(), W1, W2)
    with pytest.raises(moe.MoEError, match="INVALID"):
        moe.gated_ffn(x[:0], W1, W2, out=torch.empty(0, 128, device="cuda", dtype=BF16), workspace=ffn.workspace)
    with pytest.raises(moe.MoEError, match="UNSUPPORTED"):
        moe.GatedFFN(torch.zeros(8, 12, device="cuda", dtype=BF16), torch.zeros(12, 4, device="cuda", dtype=BF16))
    both = torch.zeros(41, 128, device="cuda", dtype=BF16)
    with pytest.raises(moe.MoEError, match="INVALID"):      # shifted by a row
        moe.gated_ffn(x, W1, W2, "gelu", add=both[:40], out=both[1:])
    with pytest.raises(moe.MoEError, match="WORKSPACE"):
        moe.gated_ffn(x, W1, W2, "gelu", workspace=ffn.workspace[:4000])
    pre = torch.empty(40, 128, device="cuda", dtype=BF16)
    with pytest.raises(TypeError, match="dW2"):             # one type for both
        moe.gated_ffn_backward(x, pre, dy, W1, W2, "gelu",
                               out=moe.GatedFFNGrads(None, torch.empty(128, 128, device="cuda"), torch.empty_like(W2)))
    with pytest.raises(moe.MoEError, match="INVALID"):      # a sum for a dx that is not wanted
        moe.gated_ffn_backward(x, pre, dy, W1, W2, "gelu", add=add, out=moe.GatedFFNGrads(None, torch.empty_like(W1)))
    assert moe.device_status() == 0
