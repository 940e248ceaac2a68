"""The operators together: a layer routed by scores, alone against the oracle,
and inside a residual stream with its norms, gate and gradient clipping."""
import numpy as np
import pytest
import torch

import dropless_moe_expert_gb300 as moe
import oracle
from oracle import operators as op
from workloads import Shape, make_tokens, make_weights

from _helpers import check_output, to_np

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16

CASES = [
    (Shape(T=300, d=256, E=64, K=6, f=128), moe.RouteRule("sigmoid", 8, 4, 2, True, 2.5), True),
    (Shape(T=129, d=128, E=16, K=4, f=192, bias="normal_0.5"), moe.RouteRule("sigmoid", 1, 1, 1, False, 1.0), False),
    (Shape(T=200, d=192, E=32, K=4, f=128), moe.RouteRule("softmax", 4, 2, 1, True, 1.5), True),
    (Shape(T=1, d=128, E=8, K=2, f=64), moe.RouteRule("sigmoid", 2, 1, 2, True, 1.0), True),
    (Shape(T=1500, d=128, E=2, K=2, f=192), moe.RouteRule("softmax", 1, 1, 1, True, 1.0), False),
]


def _layer(s, rule, bias):
    w = make_weights(s, seed=0, device="cpu")
    sel = (0.05 * torch.randn(s.E, generator=torch.Generator().manual_seed(9))).cuda() if bias else None
    return w, moe.MoELayer(w.Wr.cuda(), w.bias.cuda(), w.W1.cuda(), w.W2.cuda(), s.K, s.T, rule=rule, sel_bias=sel), sel


@pytest.mark.parametrize("s,rule,bias", CASES, ids=str)
def test_layer_routed_by_scores(s, rule, bias):
    """y and the gradients against the oracle for the choice the GPU made (the
    choice itself: tests/test_route_scored.py), with the layer's tolerances."""
    w, layer, sel = _layer(s, rule, bias)
    x = make_tokens(s, seed=1, device="cpu")
    y = layer(x.cuda(), save_preact=True)
    v = layer.views(s.T)
    direct = moe.route_scored(v["logits"].clone(), s.K, rule, sel)
    for k in ("topk_idx", "topk_w", "counts", "offsets", "row_of", "src_tok"):
        assert torch.equal(getattr(direct, k), v[k]), k
    idx = to_np(v["topk_idx"])
    gate = op.route_scored_weights(to_np(v["logits"]), idx, rule.score, rule.renorm, rule.scale)
    xs, Wr, W1, W2 = (t.float().numpy() for t in (x, w.Wr, w.W1, w.W2))
    _, offsets = oracle.expert_counts(idx, s.E)
    src_tok, row_of = oracle.dispatch_order(idx, s.E)
    _, y_perm = oracle.grouped_mlp(oracle.permute(xs, src_tok), offsets, W1, W2)
    check_output(to_np(y), oracle.combine(y_perm, row_of, gate))
    # the unfused and the fused forward agree with the training one
    assert torch.equal(layer(x.cuda()), y)

    layer(x.cuda(), save_preact=True)
    dy = torch.randn((s.T, s.d), generator=torch.Generator().manual_seed(3)).to(BF16)
    g = layer.backward(x.cuda(), dy.cuda())
    ref = oracle.backward(xs, Wr, w.bias.numpy(), W1, W2, s.K, dy.float().numpy(),
                          dict(idx=idx, w=gate, offsets=offsets, src_tok=src_tok, row_of=row_of))
    dL, _ = op.route_scored_backward(to_np(v["logits"]), idx, ref["dw"], rule.score, rule.renorm, rule.scale)
    dx = ref["dx"] + (dL - ref["dL"]) @ Wr.astype(np.float64).T
    for name, want in (("dx", dx), ("dW1", ref["dW1"]), ("dW2", ref["dW2"])):
        n = np.linalg.norm(want)
        assert np.linalg.norm(to_np(g[name]).astype(np.float64) - want) <= 1e-2 * (n if n else 1.0), name
    # the router's gradients cancel: bounded by the terms that each sums (bf16 y_perm behind dw)
    _, row_of_ = oracle.dispatch_order(idx, s.E)
    dwm = np.einsum("tkc,tc->tk", np.abs(ref["y_perm"])[row_of_], np.abs(dy.float().numpy().astype(np.float64)))
    _, mag = op.route_scored_backward(to_np(v["logits"]), idx, dwm, rule.score, rule.renorm, rule.scale)
    assert np.all(np.abs(to_np(g["dbias"]) - dL.sum(0)) <= 2.0 ** -5 * mag.sum(0) + 1e-6 * mag.sum(0).max())
    S = np.abs(xs.astype(np.float64)).T @ mag
    assert np.all(np.abs(to_np(g["dWr"]) - xs.astype(np.float64).T @ dL) <= 2.0 ** -5 * S + 1e-6 * S.max())


def test_layer_with_one_renormalised_choice():
    """K = 1 with renorm: the router gets no gradient, and dx only that of the expert."""
    s = Shape(T=200, d=128, E=8, K=1, f=64)
    w, layer, _ = _layer(s, moe.RouteRule("sigmoid", 2, 1, 2, True, 1.7), True)
    x = make_tokens(s, seed=1, device="cpu").cuda()
    y = layer(x, save_preact=True)
    assert bool((layer.views(s.T)["topk_w"] == 1.7).all())
    g = layer.backward(x, y)
    assert not bool(g["dWr"].any()) and not bool(g["dbias"].any()) and bool(g["dx"].any())


def test_raw_softmax_layer_has_no_backward():
    s = Shape(T=64, d=128, E=8, K=2, f=64)
    _, layer, _ = _layer(s, moe.RouteRule("softmax", renorm=False), False)
    x = make_tokens(s, seed=1, device="cpu").cuda()
    layer(x, save_preact=True)
    with pytest.raises(moe.MoEError, match="UNSUPPORTED"):
        layer.backward(x, x)


@pytest.mark.parametrize("dt", [torch.float32, BF16])
def test_two_blocks_and_clipping(dt):
    """Two blocks in a stream, forward and backward, equal the steps called one
    by one (each checked against the oracle elsewhere) bit for bit; then the
    gradients of both are clipped by their common norm."""
    s = Shape(T=257, d=256, E=16, K=4, f=128)
    rule = moe.RouteRule("sigmoid", 4, 2, 2, True, 2.0)
    g = torch.Generator(device="cuda").manual_seed(0)
    vec = [1 + 0.1 * torch.randn(s.d, generator=g, device="cuda") for _ in range(5)]
    layers = [_layer(s, rule, True)[1] for _ in range(2)]
    blocks = [moe.MoEBlock(layers[0], vec[0], vec[1], 0.3 * vec[2], 0.9), moe.MoEBlock(layers[1], vec[3], vec[4], None)]
    r0 = torch.randn(s.T, s.d, generator=g, device="cuda").to(dt)
    a = blocks[0](r0, next_gamma=vec[3], save=True)
    b = blocks[1](a.r, pre=a, save=True)
    dr = torch.randn(s.T, s.d, generator=g, device="cuda").to(dt)
    gb = blocks[1].backward(dr)
    ga = blocks[0].backward(gb["dr"], gb["dn"])

    n0 = moe.norm_residual(r0, gamma_pre=vec[0])
    l0, l1 = (_layer(s, rule, True)[1] for _ in range(2))
    y0 = l0(n0.n, save_preact=True)
    a2 = moe.norm_residual(r0, y0, gamma_post=vec[1], gate=0.3 * vec[2], gamma_pre=vec[3], res_scale=0.9)
    y1 = l1(a2.n, save_preact=True)
    b2 = moe.norm_residual(a2.r, y1, gamma_post=vec[4])
    assert torch.equal(a.r, a2.r) and torch.equal(a.n, a2.n) and torch.equal(b.r, b2.r) and b.n is None
    h1 = moe.norm_residual_backward(b2.r, dr, None, y1, gamma_post=vec[4], rstd_post=b2.rstd_post)
    k1 = l1.backward(a2.n, h1.dy)
    h0 = moe.norm_residual_backward(a2.r, h1.dr, k1["dx"], y0, gamma_post=vec[1], gate=0.3 * vec[2], gamma_pre=vec[3],
                                    res_scale=0.9, rstd_post=a2.rstd_post, rstd_pre=a2.rstd_pre)
    k0 = l0.backward(n0.n, h0.dy)
    e = moe.norm_residual_backward(r0, h0.dr, k0["dx"], gamma_pre=vec[0], rstd_pre=n0.rstd_pre)
    assert torch.equal(gb["dr"], h1.dr) and torch.equal(gb["dn"], k1["dx"]) and torch.equal(gb["dgamma_post"], h1.dgamma_post)
    assert torch.equal(ga["dr"], e.dr) and ga["dn"] is None and torch.equal(ga["dgamma_pre"], e.dgamma_pre)
    assert torch.equal(ga["dgate"], h0.dgate) and torch.equal(ga["dnext_gamma"], h0.dgamma_pre)
    for k in ("dW1", "dW2", "dWr", "dbias"):
        assert torch.equal(ga[k], k0[k]) and torch.equal(gb[k], k1[k]), k

    params = [t for q in (ga, gb) for k, t in q.items() if k not in ("dr", "dn") and t is not None]
    raw = [to_np(t).astype(np.float64) for t in params]
    norm = float(moe.GradClipper(params)(1.0))
    ref = op.grad_norm(raw)
    assert abs(norm - ref) <= 128 * 2.0 ** -24 * ref and ref > 1.0
    assert abs(op.grad_norm([to_np(t) for t in params]) - 1.0) <= 1e-4
    with pytest.raises(RuntimeError, match="save"):
        moe.MoEBlock(layers[0], vec[0]).backward(dr)


def test_step_in_a_graph():
    """Forward, backward and clipping of a block captured once and replayed on
    another stream: the bits of an eager step on the same tokens."""
    s = Shape(T=300, d=128, E=32, K=4, f=128)
    rule = moe.RouteRule("sigmoid", 4, 2, 2)
    _, layer, _ = _layer(s, rule, True)
    block = moe.MoEBlock(layer, torch.ones(s.d, device="cuda"), torch.ones(s.d, device="cuda"))
    r = torch.randn(s.T, s.d, device="cuda")
    dr = torch.randn(s.T, s.d, device="cuda")

    def step():
        out = block(r, save=True)
        g = block.backward(dr)
        names = [k for k in g if g[k] is not None and k != "dr"]
        norm = moe.GradClipper([g[k] for k in names])(0.5)
        return [out.r, g["dr"], norm] + [g[k] for k in names]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    r.normal_()
    dr.normal_()
    graph.replay()
    torch.cuda.synchronize()
    assert moe.device_status() == 0
    got = [t.clone() for t in got]
    for a, b in zip(got, step()):
        assert torch.equal(a, b)
