"""The Python objects of the operators around the layer: their copies, buffers
that are replaced or used in another form, streams, and a layer that several
blocks share."""
import copy
import ctypes
import dataclasses
import gc
import pickle

import pytest
import torch

import dropless_moe_expert_gb300 as moe


# ------------------------------------------------------------------ RouteRule
def _fields(struct):
    return tuple(getattr(struct, n) for n, _ in struct._fields_)


@pytest.mark.parametrize("how", [copy.copy, copy.deepcopy, dataclasses.replace, lambda r: pickle.loads(pickle.dumps(r))],
                         ids=["copy", "deepcopy", "replace", "pickle"])
def test_copies_of_a_rule_pass_their_own_values(how):
    """What a copy hands to the library is its own struct, also when the original is gone."""
    original = moe.RouteRule("softmax", 8, 4, 2, True, 2.5)
    rule = how(original)
    assert rule == original
    del original
    gc.collect()
    others = [moe.RouteRule("sigmoid", 1, 1, 1, False, 9.0) for _ in range(64)]   # may take the freed memory
    assert rule._c == ctypes.addressof(rule._struct)
    assert _fields(moe._RouteRule.from_address(rule._c)) == (1, 8, 4, 2, 1, 2.5)
    assert len(others) == 64


# ------------------------------------------------------------------ RouteBuffers
ROUTING = ("topk_idx", "topk_w", "counts", "offsets", "row_of", "src_tok")


@pytest.fixture
def called(monkeypatch):
    """The arguments of the library's calls, which are recorded instead of made; tensors may lie on the CPU."""
    calls = []

    class Recorder:
        def __getattr__(self, name):
            if name.endswith("_size"):
                return getattr(real, name)
            return lambda *a: calls.append((name, a)) or 0

    real = moe.lib
    monkeypatch.setattr(moe, "lib", Recorder())
    monkeypatch.setattr(moe, "_need", lambda t, dtype, shape, name: t)
    monkeypatch.setattr(moe, "_in", lambda t, dtype, shape, name: t.data_ptr())
    monkeypatch.setattr(moe, "_stream_of", lambda t, stream=None: 0)
    return calls


def test_buffers_pass_the_addresses_of_their_own_tensors(called):
    """Copies of the buffers, and buffers one of whose tensors was replaced or given other memory."""
    logits, rule = torch.zeros(40, 16), moe.RouteRule()
    first = moe.RouteBuffers(40, 16, 2, "cpu")
    moe.route_scored(logits, 2, rule, buffers=first)
    replaced = moe.RouteBuffers(40, 16, 2, "cpu")
    moe.route_scored(logits, 2, rule, buffers=replaced)
    replaced.routing.topk_w = torch.empty(40, 2)
    replaced.routing.row_of.data = torch.empty(40, 2, dtype=torch.int32)
    replaced.workspace = torch.empty(replaced.workspace.numel() + 16, dtype=torch.uint8)
    for b in (copy.deepcopy(first), pickle.loads(pickle.dumps(first)), replaced, first):
        called.clear()
        r = moe.route_scored(logits, 2, rule, buffers=b)
        (_, args), = called
        assert r is b.routing
        assert args[6:14] == (*[getattr(r, k).data_ptr() for k in ROUTING], b.workspace.data_ptr(), b.workspace.numel())


@pytest.mark.gpu
def test_buffers_that_are_copied_or_replaced():
    logits, rule = torch.randn(700, 64, device="cuda"), moe.RouteRule("sigmoid", 8, 4, 2)
    first = moe.RouteBuffers(700, 64, 6)
    kept = {k: getattr(moe.route_scored(logits, 6, rule, buffers=first), k).clone() for k in ROUTING}
    other = copy.deepcopy(first)
    flipped = {k: getattr(moe.route_scored(-logits, 6, rule), k) for k in ROUTING}
    moe.route_scored(-logits, 6, rule, buffers=other)
    for k in ROUTING:
        assert torch.equal(getattr(first.routing, k), kept[k]) and torch.equal(getattr(other.routing, k), flipped[k])
    first.routing.topk_idx = torch.empty_like(kept["topk_idx"])
    assert torch.equal(moe.route_scored(-logits, 6, rule, buffers=first).topk_idx, flipped["topk_idx"])
    first.routing.topk_w.data = torch.empty(10, 6, device="cuda")
    with pytest.raises(ValueError, match="topk_w"):
        moe.route_scored(logits, 6, rule, buffers=first)
    other.workspace = torch.empty(16, dtype=torch.uint8, device="cuda")
    with pytest.raises(moe.MoEError, match="WORKSPACE"):
        moe.route_scored(logits, 6, rule, buffers=other)
    with pytest.raises(ValueError, match="CUDA"):
        moe.route_scored(logits, 6, rule, buffers=moe.RouteBuffers(700, 64, 6, "cpu"))


# ------------------------------------------------------------------ NormResidual
def test_buffers_keep_their_stream_in_a_call_without_y(called):
    """The form without y leaves ``out`` as it was; a later call with y does not write the earlier one's input."""
    T, d = 5, 64
    r, y, g = torch.zeros(T, d), torch.zeros(T, d, dtype=torch.bfloat16), torch.ones(d)
    out = moe.NormResidual.empty(T, d, torch.float32, post=False, device="cpu")
    own = out.r
    o = moe.norm_residual(r, gamma_pre=g, out=out)
    assert o.r is r and o.n is out.n and o.rstd_pre is out.rstd_pre and out.r is own
    o = moe.norm_residual(r, y, gamma_pre=g, out=out)
    assert o is out and called[-1][1][11] == own.data_ptr()


@pytest.mark.gpu
def test_one_buffer_for_two_forms():
    T, d = 33, 320
    r, g = torch.randn(T, d, device="cuda"), torch.rand(d, device="cuda")
    y = torch.randn(T, d, device="cuda").to(torch.bfloat16)
    raw, out = r.clone(), moe.NormResidual.empty(T, d, torch.float32, post=False)
    n = moe.norm_residual(r, gamma_pre=g, out=out).n.clone()
    with_y = moe.norm_residual(r, y, gamma_pre=g, out=out)
    ref = moe.norm_residual(raw, y, gamma_pre=g)
    assert torch.equal(r, raw) and torch.equal(with_y.r, ref.r) and torch.equal(with_y.n, ref.n)
    assert torch.equal(moe.norm_residual(r, gamma_pre=g, out=out).n, n) and torch.equal(with_y.r, ref.r)


@pytest.mark.gpu
def test_norm_buffers_with_other_memory():
    """Buffers that were accepted once and then given other memory: written there where it fits, else refused."""
    T, d, bf = 40, 256, torch.bfloat16
    r, g = torch.randn(T, d, device="cuda"), torch.rand(d, device="cuda")
    y = torch.randn(T, d, device="cuda").to(bf)
    ref = moe.norm_residual(r, y, gamma_pre=g)
    out = moe.NormResidual.empty(T, d, torch.float32, post=False)
    moe.norm_residual(r, y, gamma_pre=g, out=out)
    out.n.data = torch.zeros(T, d, dtype=bf, device="cuda")
    out.r.set_(torch.zeros(2 * T, d, device="cuda")[T:])
    moe.norm_residual(r, y, gamma_pre=g, out=out)
    assert torch.equal(out.n, ref.n) and torch.equal(out.r, ref.r)
    twin = copy.deepcopy(out)
    moe.norm_residual(2 * r, y, gamma_pre=g, out=twin)
    assert torch.equal(out.r, ref.r) and not torch.equal(twin.r, ref.r)
    dr = torch.randn(T, d, device="cuda")
    grads = moe.NormResidualGrads.empty(T, d, torch.float32, post=False)

    def backward(o):
        return moe.norm_residual_backward(ref.r, dr, y, y, gamma_pre=g, rstd_pre=ref.rstd_pre, out=o)

    gref = moe.norm_residual_backward(ref.r, dr, y, y, gamma_pre=g, rstd_pre=ref.rstd_pre)
    backward(grads)
    grads.dgamma_pre.data = torch.zeros(d, device="cuda")
    grads.workspace = None
    backward(grads)
    assert torch.equal(grads.dgamma_pre, gref.dgamma_pre) and torch.equal(grads.dy, gref.dy)


@pytest.mark.gpu
def test_norm_buffers_are_refused_once_they_do_not_fit():
    """The same objects, now shorter, of another type or on the host: no call reads or writes them."""
    T, d, bf = 40, 256, torch.bfloat16
    r, g = torch.randn(T, d, device="cuda"), torch.rand(d, device="cuda")
    y = torch.randn(T, d, device="cuda").to(bf)
    ref = moe.norm_residual(r, y, gamma_pre=g)
    before = moe.launch_count()
    for name, other, what in (("n", torch.zeros(3, d, dtype=bf, device="cuda"), ValueError),
                              ("r", torch.zeros(T, d, dtype=bf, device="cuda"), TypeError),
                              ("rstd_pre", torch.zeros(T - 1, device="cuda"), ValueError)):
        out = moe.NormResidual.empty(T, d, torch.float32, post=False)
        out._pointers((T, d, torch.float32, True, False, True))      # as a call does
        getattr(out, name).data = other
        with pytest.raises(what, match="out." + name):
            moe.norm_residual(r, y, gamma_pre=g, out=out)
    with pytest.raises(ValueError, match="CUDA"):
        moe.norm_residual(r, y, gamma_pre=g, out=moe.NormResidual.empty(T, d, torch.float32, device="cpu"))
    for name, other in (("dy", torch.zeros(T, 2 * d, dtype=bf, device="cuda")[:, :d]), ("dr", torch.zeros(1, device="cuda")),
                        ("workspace", torch.zeros(1 << 20, dtype=torch.uint8)),
                        ("workspace", torch.zeros(1 << 20, device="cuda")),
                        ("workspace", torch.zeros(4096, dtype=torch.uint8, device="cuda"))):
        grads = moe.NormResidualGrads.empty(T, d, torch.float32, post=False)
        setattr(grads, name, other)
        with pytest.raises((ValueError, TypeError, moe.MoEError)):
            moe.norm_residual_backward(ref.r, r, y, y, gamma_pre=g, rstd_pre=ref.rstd_pre, out=grads)
    assert moe.launch_count() == before


def test_norm_buffers_are_checked_again(called, monkeypatch):
    """The check runs once for buffers that stay as they are, and again for those that were given other memory."""
    checked = []
    monkeypatch.setattr(moe, "_need", lambda t, dtype, shape, name: checked.append(name) or t)
    T, d, f32 = 4, 64, torch.float32
    r, y, g = torch.zeros(T, d), torch.zeros(T, d, dtype=torch.bfloat16), torch.ones(d)
    out = moe.NormResidual.empty(T, d, f32, post=False, device="cpu")
    grads = moe.NormResidualGrads.empty(T, d, f32, post=False, device="cpu")

    def call():
        checked.clear()
        moe.norm_residual(r, y, gamma_pre=g, out=out)
        moe.norm_residual_backward(r, r, y, y, gamma_pre=g, rstd_pre=g[:T], out=grads)
        return set(checked)

    assert {"out.r", "out.n", "out.rstd_pre", "out.dr", "out.dy", "out.dgamma_pre", "out.workspace"} <= call()
    assert not call()
    out.n.data = torch.zeros(T - 1, d, dtype=torch.bfloat16)
    assert "out.n" in call() and not call()
    grads.dy.resize_(8 * T, d)
    assert "out.dy" in call() and not call()
    grads.workspace = torch.zeros(16, dtype=torch.uint8)
    assert "out.workspace" in call()


# ------------------------------------------------------------------ GradClipper
def test_clipper_passes_where_the_tensors_lie(called):
    """Gradients and outputs that were given other memory, and copies of a clipper."""
    grads = [torch.ones(n) for n in (5, 40, 0, 7)]
    outs = [torch.ones(n) for n in (5, 40, 0, 7)]

    def check(clipper, gs, os):
        called.clear()
        clipper(1.0)
        clipper()
        (_, clip), (_, norm) = called
        for args in (clip, norm):
            assert [p or 0 for p in args[0]] == [g.data_ptr() for g in gs]
        assert (clip[1] is None) == (os is None)
        assert os is None or [p or 0 for p in clip[1]] == [o.data_ptr() for o in os]
        assert clip[6] == norm[4] == clipper.norm.data_ptr()

    beside, in_place = moe.GradClipper(grads, outs), moe.GradClipper(grads)
    check(beside, grads, outs)
    check(in_place, grads, None)
    grads[1].data = torch.ones(40)
    grads[3].set_(torch.ones(20)[3:10])
    outs[0].data = torch.ones(5)
    check(beside, grads, outs)
    check(in_place, grads, None)
    for twin in (copy.copy(beside), copy.deepcopy(beside), pickle.loads(pickle.dumps(beside))):
        check(twin, twin.grads, twin.outs)
    assert [tuple(g.shape) for g in copy.deepcopy(in_place).grads] == [(5,), (40,), (0,), (7,)]


def test_clipper_holds_the_memory_whose_address_it_keeps(called):
    """Memory that a call went by is not given to another tensor while its address is kept."""
    grads = [torch.ones(1 << 20)]
    clipper = moe.GradClipper(grads)
    old = grads[0].data_ptr()
    grads[0].data = torch.ones(1 << 20)
    later = [torch.empty(1 << 20) for _ in range(4)]
    assert all(t.data_ptr() != old for t in later)


@pytest.mark.gpu
def test_clipper_follows_its_tensors():
    g = torch.Generator(device="cuda").manual_seed(3)
    grads = [torch.randn(n, generator=g, device="cuda").to(k) for n, k in ((5000, torch.float32), (333, torch.bfloat16))]
    clipper = moe.GradClipper(grads)
    clipper(0.5)
    old = grads[0].detach()
    kept = old.clone()
    fresh = torch.randn(5000, generator=g, device="cuda")
    grads[0].data = fresh.clone()
    want = [fresh.clone(), grads[1].clone()]
    ref = moe.GradClipper(want)(0.5)
    assert torch.equal(clipper(0.5), ref) and all(torch.equal(a, b) for a, b in zip(grads, want))
    assert torch.equal(old, kept)                       # the memory that the gradient had left
    twin = copy.deepcopy(clipper)
    norm = clipper().clone()
    assert torch.equal(twin(), norm) and twin.grads[0].data_ptr() != grads[0].data_ptr()
    for other, what in ((torch.zeros(5, device="cuda"), ValueError), (torch.zeros(5000, 2, device="cuda")[:, 0], ValueError),
                        (torch.zeros(5000, dtype=torch.bfloat16, device="cuda"), TypeError)):
        grads[0].data = other
        with pytest.raises(what, match=r"grads\[0\]"):
            clipper(0.5)
    with pytest.raises(AttributeError):
        clipper.norm = torch.zeros(1, device="cuda")


def test_clipper_refuses_tensors_that_are_written_over(called):
    """What a call writes overlaps nothing else that it reads or writes, but an output may be its own gradient."""
    flat, other = torch.ones(100), torch.ones(100)
    a, b, c = flat[:40], flat[40:90], flat[90:]
    moe.GradClipper([a, b, c])
    moe.GradClipper([a, a, flat], [other[:40], other[40:80], torch.ones(100)])   # gradients are only read
    moe.GradClipper([a, b], [a, b])                                              # in place, said twice
    moe.GradClipper([a, b, flat[:0]], [other[10:50], other[50:], flat[20:20]])   # nothing lies in no elements
    for grads, outs in (([a, a], None), ([flat, c], None), ([a, flat[39:60]], None), ([a], [flat[1:41]]),
                        ([a, b], [other[:40], other[39:89]]), ([a, b], [flat[50:90], other[:50]]),
                        ([a, a], [a, other[:40]]), ([a, flat], [other[:40], flat])):
        with pytest.raises(ValueError, match="overlap"):
            moe.GradClipper(grads, outs)
    clipper = moe.GradClipper([a, b])
    b.set_(flat[30:80])
    with pytest.raises(ValueError, match="overlap"):
        clipper(1.0)


# ------------------------------------------------------------------ streams
class _Side:
    cuda_stream = 7


def _small_block(device, T=24, E=8, K=2, d=128, f=64):
    g = torch.Generator(device="cpu").manual_seed(1)

    def normal(*shape):
        return torch.randn(*shape, generator=g)

    Wr, W1, W2 = normal(d, E), 0.1 * normal(E, 2 * f, d), 0.1 * normal(E, d, f)
    layer = moe.MoELayer(Wr.to(device), torch.zeros(E, device=device), W1.to(torch.bfloat16).to(device),
                         W2.to(torch.bfloat16).to(device), K, T, rule=moe.RouteRule("sigmoid", 4, 2, 2))
    block = moe.MoEBlock(layer, torch.ones(d, device=device), torch.ones(d, device=device))
    return block, normal(T, d).to(device), normal(T, d).to(device)


def test_a_call_on_a_stream_allocates_there(called, monkeypatch):
    """What a call with ``stream`` allocates belongs to that stream, and is not reused before the current one has passed."""
    inside, made, recorded = [], [], set()
    empty = torch.empty

    class Inside:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            inside.append(self.stream)

        def __exit__(self, *a):
            inside.pop()

    def record(*shape, **kw):
        t = empty(*shape, **kw)
        made.append((bool(inside), t))
        return t

    monkeypatch.setattr(torch.cuda, "stream", Inside)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: _Side())
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: recorded.add(id(t)))
    block, r, dr = _small_block("cpu")
    bf = torch.bfloat16
    logits, rule, side = torch.zeros(24, 8), moe.RouteRule(), _Side()
    calls = [lambda s: moe.route_scored(logits, 2, rule, stream=s),
             lambda s: moe.route_scored_backward(logits, torch.zeros(24, 2, dtype=torch.int32), logits[:, :2], rule, stream=s),
             lambda s: moe.norm_residual(r, r.to(bf), gamma_pre=r[0], stream=s),
             lambda s: moe.norm_residual_backward(r, r, r.to(bf), r.to(bf), gamma_pre=r[0], rstd_pre=r[:, 0], stream=s),
             lambda s: moe.norm_residual_backward(r, r, None, r.to(bf), stream=s, out=moe.NormResidualGrads(r, r.to(bf))),
             lambda s: moe.route(logits, 2, stream=s), lambda s: block(r, save=True, stream=s),
             lambda s: block.backward(dr, stream=s)]
    monkeypatch.setattr(torch, "empty", record)
    for call in calls:
        made.clear()
        recorded.clear()
        call(side)
        assert made and all(on for on, _ in made) and {id(t) for _, t in made} <= recorded
        made.clear()
        call(None)
        assert not any(on for on, _ in made)


@pytest.mark.gpu
def test_a_block_on_a_stream_keeps_its_memory():
    """Work of the current stream that allocates while a side stream is late gets none of the memory that is in use there."""
    block, r, dr = _small_block("cuda", T=700, d=256)
    want = block(r, save=True)
    wantg = block.backward(dr)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    sizes = sorted({t.numel() * t.element_size() for t in [want.r, want.rstd_post, r.to(torch.bfloat16), *wantg.values()]
                    if t is not None} | {int(moe.lib.moe_norm_residual_backward_workspace_size(700, 256)), 1 << 20})
    rule, logits = moe.RouteRule(), torch.randn(5000, 64, device="cuda")
    routed = moe.route_scored(logits, 6, rule)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)          # about ten milliseconds
    out = block(r, save=True, stream=side)
    grads = block.backward(dr, stream=side)
    again = moe.route_scored(logits, 6, rule, stream=side)
    filled = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(12)]
    filled += [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in range(512, 8192, 512)]
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out.r, want.r)
    for k, v in wantg.items():
        assert (v is None and grads[k] is None) or torch.equal(grads[k], v), k
    for k in ROUTING:
        assert torch.equal(getattr(again, k), getattr(routed, k)), k
    assert all(bool((t == 255).all()) for t in filled)


# ------------------------------------------------------------------ blocks that share a layer
def test_backward_refuses_a_layer_that_has_run_since(called, monkeypatch):
    """The layer keeps one call's routing and activations: a later call of it, by another block or by itself, is noticed."""
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: _Side())
    block, r, dr = _small_block("cpu")
    other = moe.MoEBlock(block.layer, block.gamma_pre)
    for run in (lambda: other(r), lambda: block.layer(r.to(torch.bfloat16)), lambda: block.layer(r.to(torch.bfloat16), save_preact=True)):
        block(r, save=True)
        run()
        called.clear()
        with pytest.raises(RuntimeError, match="layer"):
            block.backward(dr)
        assert not called
    block(r, save=True)
    block.backward(dr)
    block.backward(dr)      # the saved call may be differentiated again


@pytest.mark.gpu
def test_blocks_that_share_a_layer():
    block, r, dr = _small_block("cuda")
    other = moe.MoEBlock(block.layer, 2 * block.gamma_pre)
    a = block(r, save=True)
    want = block.backward(dr)
    block(r, save=True)
    b = other(a.r, save=True)
    with pytest.raises(RuntimeError, match="layer"):
        block.backward(dr)
    other.backward(dr)
    assert torch.equal(block(r, save=True).r, a.r) and not torch.equal(a.r, b.r)
    for k, v in block.backward(dr).items():
        assert (v is None and want[k] is None) or torch.equal(v, want[k]), k


def test_a_norm_of_another_eps_is_refused(called, monkeypatch):
    """A block takes the norm that the block before it left only where that used this block's eps."""
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: _Side())
    first, r, _ = _small_block("cpu")
    same, other = (moe.MoEBlock(first.layer, first.gamma_pre, eps=e) for e in (1e-6, 1e-5))
    n = first(r, next_gamma=same.gamma_pre)
    same(n.r, pre=n)
    with pytest.raises(ValueError, match="eps"):
        other(n.r, pre=n)
    own = moe.norm_residual(r, gamma_pre=other.gamma_pre, eps=1e-5, out=moe.NormResidual.empty(24, 128, y=False, post=False,
                                                                                            device="cpu"))
    other(r, pre=own)
    with pytest.raises(ValueError, match="eps"):
        same(r, pre=copy.copy(own))
    same(r, pre=moe.NormResidual(r, own.n))     # the caller's own


def test_a_block_that_has_no_backward_refuses_to_save_for_it(called, monkeypatch):
    """Raw softmax scores: the layer's backward does not take them, so a training forward of a block stops before it runs."""
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: _Side())
    block, r, _ = _small_block("cpu")
    block.layer.rule = moe.RouteRule("softmax", renorm=False)
    with pytest.raises(ValueError, match="softmax"):
        block(r, save=True)
    assert not called
    block(r)
    for rule in (moe.RouteRule("softmax"), moe.RouteRule("sigmoid", renorm=False), None):
        block.layer.rule = rule
        block(r, save=True)
