"""The operators around the layer refuse bad arguments on the host, before
anything is launched (so these run without a GPU)."""
import ctypes

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


def _rule(moe, **kw):
    base = dict(score=0, n_group=4, topk_group=2, group_top=2, renorm=1, scale=1.0)
    return ctypes.byref(moe._RouteRule(*{**base, **kw}.values()))


def _route(moe, rule, T=8, E=64, K=4, at={}, ws=BIG):
    p = {**dict(l=FAKE, b=None, i=FAKE, w=FAKE, c=FAKE, o=FAKE, r=FAKE, s=FAKE, ws=FAKE), **at}
    return moe.lib.moe_route_scored(p["l"], p["b"], T, E, K, rule, p["i"], p["w"], p["c"], p["o"], p["r"], p["s"],
                                    p["ws"], ws, None)


def test_route_scored_refusals(moe):
    r = _rule(moe)
    for bad in (dict(score=2), dict(score=-1), dict(n_group=0), dict(n_group=3), dict(topk_group=0), dict(topk_group=5),
                dict(group_top=0), dict(group_top=3), dict(scale=float("nan")), dict(scale=float("inf"))):
        assert _route(moe, _rule(moe, **bad)) == 1, bad
        assert moe.lib.moe_route_scored_backward(FAKE, FAKE, FAKE, 8, 64, 4, _rule(moe, **bad), FAKE, None) == 1
    assert _route(moe, None) == 1
    assert _route(moe, _rule(moe, n_group=16, topk_group=1), K=5) == 1      # 4 experts stay open
    assert _route(moe, r, T=0) == 1 and _route(moe, r, K=0) == 1 and _route(moe, r, K=65) == 1
    assert _route(moe, r, E=512) == 2 and _route(moe, _rule(moe, n_group=1, topk_group=1), K=17) == 2
    for name in ("l", "i", "w", "c", "o", "r", "s", "ws"):
        assert _route(moe, r, at={name: None}) == 1 and _route(moe, r, at={name: FAKE + 2}) == 1
    assert _route(moe, r, at={"b": FAKE + 1}) == 1 and _route(moe, r, at={"ws": FAKE + 8}) == 1
    assert moe.lib.moe_route_scored_workspace_size(0, 64, 4) == 0
    assert moe.lib.moe_route_scored_workspace_size(8, 512, 4) == 0
    assert _route(moe, r, T=1000, ws=moe.lib.moe_route_scored_workspace_size(1000, 64, 4) - 16) == 3
    for args in ((None, FAKE, FAKE), (FAKE, None, FAKE), (FAKE, FAKE, None), (FAKE, FAKE + 2, FAKE)):
        assert moe.lib.moe_route_scored_backward(*args, 8, 64, 4, r, FAKE, None) == 1
    assert moe.lib.moe_route_scored_backward(FAKE, FAKE, FAKE, 8, 64, 4, r, None, None) == 1
    assert moe.lib.moe_route_scored_backward(FAKE, FAKE, FAKE, 0, 64, 4, r, FAKE, None) == 1
    with pytest.raises(ValueError, match="score"):
        moe.RouteRule(score="tanh")
    with pytest.raises(ValueError, match="rule"):
        moe.MoELayer(None, None, None, None, 2, 8, sel_bias=torch.zeros(8))


def test_scored_layer_refusals(moe):
    L, r = moe.lib, _rule(moe)
    dims = (64, 128, 64, 4, 64)
    nf, nb = L.moe_forward_workspace_size(*dims), L.moe_backward_workspace_size(*dims)

    def fwd(rule=r, bias=None, n=nf):
        return L.moe_forward_scored(FAKE, FAKE, None, bias, rule, FAKE, FAKE, *dims, FAKE, FAKE, n, None, None)

    def bwd(rule=r, n=nb):
        return L.moe_backward_scored(FAKE, FAKE, rule, FAKE, FAKE, *dims, FAKE, FAKE, nf, None, FAKE, FAKE, FAKE, FAKE,
                                     FAKE, FAKE, n, None)

    assert fwd(None) == 1 and fwd(_rule(moe, n_group=5)) == 1 and fwd(bias=FAKE + 2) == 1 and fwd(n=nf - 1) == 3
    assert bwd(None) == 1 and bwd(_rule(moe, group_top=7)) == 1 and bwd(n=nb - 1) == 3
    assert bwd(_rule(moe, score=1, renorm=0)) == 2     # raw softmax scores: a dense gradient


def _norm(moe, **kw):
    p = {**dict(r=FAKE, f32=0, y=FAKE, gp=FAKE, gate=FAKE, kind=1, a=1.0, gq=FAKE, eps=1e-6, T=4, d=128, ro=FAKE,
                n=FAKE, rp=FAKE, rq=FAKE), **kw}
    return moe.lib.moe_norm_residual(*p.values(), None)


def _norm_bwd(moe, **kw):
    p = {**dict(ro=FAKE, f32=0, y=FAKE, gp=FAKE, gate=FAKE, kind=1, a=1.0, gq=FAKE, rp=FAKE, rq=FAKE, dro=FAKE,
                dn=FAKE, T=4, d=128, dr=FAKE, dy=FAKE, dgq=FAKE, dgp=FAKE, dg=FAKE, ws=FAKE, bytes=BIG), **kw}
    return moe.lib.moe_norm_residual_backward(*p.values(), None)


def test_norm_residual_refusals(moe):
    inf, nan = float("inf"), float("nan")
    for call in (_norm, _norm_bwd):
        for bad in (dict(T=0), dict(d=0), dict(f32=2), dict(kind=3), dict(kind=0), dict(gate=None), dict(a=nan),
                    dict(a=inf), dict(y=FAKE + 8), dict(gp=FAKE + 4), dict(gq=FAKE + 4), dict(gate=FAKE + 4)):
            assert call(moe, **bad) == 1, bad
        assert call(moe, d=96) == 2 and call(moe, d=16448) == 2
        # without y there is nothing to norm, gate or scale; without gamma_pre besides, nothing to do
        assert call(moe, y=None) == 1 and call(moe, y=None, gp=None) == 1
        assert call(moe, y=None, gp=None, gate=None, kind=0, a=0.5) == 1
        assert call(moe, y=None, gp=None, gate=None, kind=0, gq=None) == 1
    for bad in (dict(eps=0.0), dict(eps=-1.0), dict(eps=nan), dict(eps=inf), dict(r=None), dict(r=FAKE + 8),
                dict(ro=None), dict(ro=FAKE + 8), dict(n=None), dict(n=FAKE + 2), dict(rp=None), dict(rq=None),
                dict(rq=FAKE + 2)):
        assert _norm(moe, **bad) == 1, bad
    for bad in (dict(dr=None), dict(dr=FAKE + 4), dict(ws=None), dict(ws=FAKE + 4), dict(dro=FAKE + 8), dict(ro=None),
                dict(dn=None), dict(rq=None), dict(dgq=None), dict(dy=None), dict(rp=None), dict(dgp=None),
                dict(dg=None), dict(dro=None, gq=None)):
        assert _norm_bwd(moe, **bad) == 1, bad
    need = moe.lib.moe_norm_residual_backward_workspace_size(4, 128)
    assert need > 0 and _norm_bwd(moe, bytes=need - 1) == 3
    for T, d in ((0, 128), (4, 100), (4, 16448)):
        assert moe.lib.moe_norm_residual_backward_workspace_size(T, d) == 0


def test_grad_clip_refusals(moe):
    L = moe.lib
    P2 = ctypes.c_void_p * 2

    def call(ptrs=(FAKE, FAKE), outs=None, sizes=(3, 5), kinds=(0, 1), n=2, max_norm=1.0, norm=FAKE, ws=FAKE, bytes=BIG):
        outs = None if outs is None else P2(*outs)
        return L.moe_grad_norm_clip(P2(*ptrs), outs, (ctypes.c_int64 * 2)(*sizes), (ctypes.c_int32 * 2)(*kinds), n,
                                    max_norm, norm, ws, bytes, None)

    for bad in (dict(n=-1), dict(max_norm=0.0), dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(norm=None),
                dict(norm=FAKE + 2), dict(ws=None), dict(ws=FAKE + 2), dict(ptrs=(None, FAKE)),
                dict(ptrs=(FAKE + 2, FAKE)), dict(ptrs=(FAKE, FAKE + 1)), dict(sizes=(-1, 5)), dict(kinds=(0, 2)),
                dict(outs=(None, FAKE)), dict(outs=(FAKE + 2, FAKE))):
        assert call(**bad) == 1, bad
    assert call(sizes=((1 << 40) + 1, 5)) == 2
    assert call(bytes=L.moe_grad_norm_workspace_size(2) - 1) == 3
    assert L.moe_grad_norm_workspace_size(-1) == 0
    assert L.moe_grad_norm(None, None, None, 2, FAKE, FAKE, BIG, None) == 1


def test_package_refuses_cpu_and_other_tensors(moe):
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="CUDA"):
        moe.route_scored(x, 2, moe.RouteRule())
    with pytest.raises(ValueError, match="CUDA"):
        moe.norm_residual(x, gamma_pre=torch.ones(64))
    with pytest.raises(TypeError, match="residual"):
        moe.norm_residual(x.half(), gamma_pre=torch.ones(64))
    with pytest.raises(ValueError, match="CUDA"):
        moe.GradClipper([x])
    with pytest.raises(TypeError, match=r"grads\[0\]"):
        moe.GradClipper([x.double()])
    with pytest.raises(ValueError, match="outs"):
        moe.GradClipper([x], outs=[])
