"""The gated feed-forward and the dropout refuse bad arguments on the host,
before anything is launched (so these run without a GPU)."""
import pytest
import torch

FAKE = 1 << 20  # a 16-byte aligned non-null address; never dereferenced (rejected first)
BIG = 1 << 40


@pytest.fixture(scope="module")
def moe():
    import dropless_moe_expert_gb300 as m
    before = m.launch_count()
    yield m
    assert m.launch_count() == before   # every call below was rejected on the host


def _ffn(moe, **kw):
    p = {**dict(x=FAKE, W1=FAKE, W2=FAKE, add=None, act=0, T=4, d=64, f=72, y=FAKE, pre=None, ws=FAKE, n=BIG), **kw}
    return moe.lib.moe_gated_ffn(*p.values(), None)


def _bwd(moe, **kw):
    p = {**dict(x=FAKE, pre=FAKE, dy=FAKE, W1=FAKE, W2=FAKE, add=None, act=0, T=4, d=64, f=72, dx=FAKE, dW1=FAKE,
                dW2=FAKE, wide=0, ws=FAKE, n=BIG), **kw}
    return moe.lib.moe_gated_ffn_backward(*p.values(), None)


def test_feed_forward_refusals(moe):
    for call in (_ffn, _bwd):
        for bad in (dict(act=-1), dict(act=4), dict(T=0), dict(T=-3), dict(d=0), dict(f=0), dict(x=FAKE + 2),
                    dict(W1=FAKE + 8), dict(W2=FAKE + 8), dict(add=FAKE + 2), dict(pre=FAKE + 4), dict(ws=FAKE + 8),
                    dict(W2=None), dict(ws=None)):
            assert call(moe, **bad) == 1, bad
        for bad in (dict(d=60), dict(f=4), dict(T=1 << 30, f=1 << 20), dict(T=1 << 30, d=1 << 20, f=8),
                    dict(f=1 << 30), dict(d=1 << 23, f=1 << 23)):
            assert call(moe, **bad) == 2, bad
    for bad in (dict(x=None), dict(W1=None), dict(y=None), dict(y=FAKE + 4)):
        assert _ffn(moe, **bad) == 1, bad
    for bad in (dict(pre=None), dict(dy=None), dict(dy=FAKE + 8), dict(dx=FAKE + 8), dict(dW1=FAKE + 8),
                dict(dW2=FAKE + 8), dict(wide=2), dict(wide=-1), dict(dx=None, dW1=None, dW2=None), dict(W1=None),
                dict(x=None), dict(dx=None, add=FAKE)):
        assert _bwd(moe, **bad) == 1, bad
    # a sum that would be read after it was written over: 4 x 64 bf16 are 512 bytes
    for shift in (16, -16, 496, -496):
        assert _ffn(moe, add=FAKE + shift) == 1 and _bwd(moe, add=FAKE + shift) == 1
    n, m = moe.lib.moe_gated_ffn_workspace_size(4, 64, 72), moe.lib.moe_gated_ffn_backward_workspace_size(4, 64, 72)
    assert n >= 4 * 72 * 2 and m >= 3 * n
    assert _ffn(moe, n=n - 1) == 3 and _bwd(moe, n=m - 1) == 3
    # dx over what the weights' gradients read beside it
    far = FAKE + (1 << 16)
    assert _bwd(moe) == 1 and _bwd(moe, x=far) == 1 and _bwd(moe, dy=far) == 1 and _bwd(moe, x=far, dy=FAKE + 496) == 1
    # the weights' gradients over each other, or over what is read beside them (dW1: 144 x 64, in fp32 36864 bytes)
    at = {k: FAKE + (i << 20) for i, k in enumerate(("x", "dy", "W1", "dx", "dW1", "dW2"))}
    for name, over in (("dW1", "x"), ("dW1", "dy"), ("dW2", "x"), ("dW2", "dy"), ("dW1", "W1"), ("dW2", "W1"),
                       ("dW2", "dW1"), ("dx", "W1"), ("dx", "dW1"), ("dx", "dW2")):
        assert _bwd(moe, **{**at, name: at[over] + 16}) == 1, (name, over)
    assert _bwd(moe, **{**at, "dW2": at["dW1"] + 36864 - 16, "wide": 1}) == 1
    for size in ((0, 64, 64), (4, 60, 64), (4, 64, 4), (4, 0, 8), (1 << 30, 64, 1 << 20)):
        assert moe.lib.moe_gated_ffn_workspace_size(*size) == 0
        assert moe.lib.moe_gated_ffn_backward_workspace_size(*size) == 0


def test_what_is_written_beside_what_is_read(moe):
    """4 tokens of 64 x 72: rows of 512 bytes in all, preact 1152, h 576, W1 18432, W2 9216."""
    at = {k: FAKE + (i << 20) for i, k in enumerate(("x", "W1", "W2", "y", "pre", "ws", "add"))}
    for a, b in ([("pre", k) for k in ("x", "W1", "W2", "y", "ws", "add")] + [("ws", k) for k in ("x", "W1", "W2", "y", "add")] +
                 [("y", "W2")]):
        for shift in (0, 16, 496):
            assert _ffn(moe, **{**at, a: at[b] + shift}) == 1, (a, b, shift)
            assert _ffn(moe, **{**at, b: at[a] + shift}) == 1, (a, b, shift)
    assert _ffn(moe, **{**at, "y": at["W2"] + 9200}) == 1 and _ffn(moe, **{**at, "pre": at["W1"] + 18416}) == 1
    at = {k: FAKE + (i << 20) for i, k in enumerate(("x", "pre", "dy", "W1", "W2", "add", "dx", "dW1", "dW2", "ws"))}
    for a, b in [("ws", k) for k in at if k != "ws"] + [("dW1", "add"), ("dW2", "add")]:
        for shift in (0, 16, 496):
            assert _bwd(moe, **{**at, a: at[b] + shift}) == 1, (a, b, shift)
            assert _bwd(moe, **{**at, b: at[a] + shift}) == 1, (a, b, shift)


def test_dropout_refusals(moe):
    def fwd(**kw):
        p = {**dict(r=FAKE, f32=0, y=FAKE, gp=None, gate=None, kind=0, a=1.0, gq=None, eps=1e-6, p=0.1, rng=FAKE, T=4,
                    d=128, ro=FAKE, n=None, rp=None, rq=None, rng_out=FAKE), **kw}
        return moe.lib.moe_norm_residual_dropout(*p.values(), None)

    def bwd(**kw):
        p = {**dict(ro=FAKE, f32=0, y=FAKE, gp=None, gate=None, kind=0, a=1.0, gq=None, p=0.1, rng=FAKE, rp=None,
                    rq=None, dro=FAKE, dn=None, T=4, d=128, dr=FAKE, dy=FAKE, dgq=None, dgp=None, dg=None, ws=FAKE,
                    n=BIG), **kw}
        return moe.lib.moe_norm_residual_dropout_backward(*p.values(), None)

    for call in (fwd, bwd):
        for bad in (dict(p=-0.1), dict(p=1.0), dict(p=float("nan")), dict(p=float("inf")), dict(p=1 - 2.0 ** -18),
                    dict(rng=None), dict(rng=FAKE + 4), dict(y=None, gq=FAKE), dict(T=0), dict(y=FAKE + 8)):
            assert call(**bad) == 1, bad
        assert call(d=96) == 2
    assert fwd(rng_out=None) == 1 and fwd(rng_out=FAKE + 4) == 1 and fwd(ro=None) == 1
    assert bwd(dy=None) == 1 and bwd(n=16) == 3


def test_package_refuses_other_tensors(moe):
    x, W1, W2 = (torch.zeros(*s, dtype=torch.bfloat16) for s in ((4, 64), (48, 64), (64, 24)))
    with pytest.raises(ValueError, match="CUDA"):
        moe.gated_ffn(x, W1, W2)
    with pytest.raises(ValueError, match="W1"):
        moe.GatedFFN(W1[:47], W2)
