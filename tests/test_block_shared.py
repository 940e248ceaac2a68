"""Blocks with a shared expert, a dense block, and dropout, together in a
stream: against the steps called one by one (each checked against the oracle
elsewhere), and in a captured training step."""
import numpy as np
import pytest
import torch

import dropless_moe_expert_gb300 as moe
from oracle import operators as op
from workloads import Shape, make_weights

from _helpers import rel_l2, to_np

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
S = Shape(T=257, d=256, E=16, K=4, f=128)
RULE = moe.RouteRule("sigmoid", 4, 2, 2, True, 2.0)


def _layer(seed=0):
    w = make_weights(S, seed=seed, device="cpu")
    return moe.MoELayer(w.Wr.cuda(), w.bias.cuda(), w.W1.cuda(), w.W2.cuda(), S.K, S.T, rule=RULE)


def _ffn(f, act, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    W1 = (torch.randn(2 * f, S.d, generator=g, device="cuda") / S.d ** 0.5).to(BF16)
    W2 = (torch.randn(S.d, f, generator=g, device="cuda") / f ** 0.5).to(BF16)
    return moe.GatedFFN(W1, W2, act, T_max=S.T)


def _vectors(n, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [1 + 0.1 * torch.randn(S.d, generator=g, device="cuda") for _ in range(n)]


@pytest.mark.parametrize("dt", [F32, BF16])
def test_two_blocks(dt):
    """A dense block, then routed experts beside a shared one, with dropout, forward and backward."""
    v = _vectors(4)
    dense, layer, shared = _ffn(520, "gelu_tanh", 0), _layer(), _ffn(136, "silu", 1)
    blocks = [moe.MoEBlock(dense, v[0], dropout=0.1), moe.MoEBlock(layer, v[1], v[2], 0.3 * v[3], shared=shared, dropout=0.2)]
    r0, dr = (torch.randn(S.T, S.d, device="cuda").to(dt) for _ in range(2))
    rng = [torch.tensor([5, k], device="cuda") for k in range(2)]
    a = blocks[0](r0, next_gamma=v[1], save=True, rng=rng[0])
    b = blocks[1](a.r, pre=a, save=True, rng=rng[1])
    state = [t.clone() for t in rng]
    for t in rng:
        t += 7          # the backward goes by what the forward drew from
    gb = blocks[1].backward(dr)
    ga = blocks[0].backward(gb["dr"], gb["dn"])

    n0 = moe.norm_residual(r0, gamma_pre=v[0])
    pre0 = torch.empty(S.T, 2 * 520, dtype=BF16, device="cuda")
    y0 = moe.gated_ffn(n0.n, dense.W1, dense.W2, "gelu_tanh", preact=pre0)
    a2 = moe.norm_residual(r0, y0, gamma_pre=v[1], dropout=0.1, rng=state[0])
    other = _layer()
    y1 = other(a2.n, save_preact=True)
    pre1 = torch.empty(S.T, 2 * 136, dtype=BF16, device="cuda")
    y1 = moe.gated_ffn(a2.n, shared.W1, shared.W2, add=y1, preact=pre1)
    gate = dict(gamma_post=v[2], gate=0.3 * v[3])
    b2 = moe.norm_residual(a2.r, y1, dropout=0.2, rng=state[1], **gate)
    assert torch.equal(a.r, a2.r) and torch.equal(a.n, a2.n) and torch.equal(b.r, b2.r)
    h1 = moe.norm_residual_backward(b2.r, dr, None, y1, rstd_post=b2.rstd_post, dropout=0.2, rng=state[1], **gate)
    k1 = other.backward(a2.n, h1.dy)
    s1 = moe.gated_ffn_backward(a2.n, pre1, h1.dy, shared.W1, shared.W2, add=k1["dx"],
                                out=moe.GatedFFNGrads.empty(S.T, S.d, 136, F32))
    h0 = moe.norm_residual_backward(a2.r, h1.dr, s1.dx, y0, gamma_pre=v[1], rstd_pre=a2.rstd_pre, dropout=0.1, rng=state[0])
    s0 = moe.gated_ffn_backward(n0.n, pre0, h0.dy, dense.W1, dense.W2, "gelu_tanh",
                                out=moe.GatedFFNGrads.empty(S.T, S.d, 520, F32))
    e = moe.norm_residual_backward(r0, h0.dr, s0.dx, gamma_pre=v[0], rstd_pre=n0.rstd_pre)
    assert torch.equal(gb["dn"], s1.dx) and torch.equal(gb["dr"], h1.dr) and torch.equal(gb["dgate"], h1.dgate)
    assert torch.equal(gb["shared_dW1"], s1.dW1) and torch.equal(gb["shared_dW2"], s1.dW2)
    for k in ("dW1", "dW2", "dWr", "dbias"):
        assert torch.equal(gb[k], k1[k]), k
    assert torch.equal(ga["dW1"], s0.dW1) and torch.equal(ga["dW2"], s0.dW2) and torch.equal(ga["dr"], e.dr)
    assert torch.equal(ga["dgamma_pre"], e.dgamma_pre) and "dWr" not in ga and ga["dn"] is None

    # without rng nothing is dropped
    quiet = blocks[0](r0, save=True)
    assert quiet.rng is None and torch.equal(quiet.r, moe.norm_residual(r0, y0).r)
    assert bool((blocks[0].backward(dr)["dr"] != 0).any())


def test_a_dense_block_against_the_oracle():
    """r' and the gradients of a dense block with dropout from end to end, each within the bf16 roundings on the
    way: n, h, y and r' forward, dy, da, n and dx backward, each 2^-8 at most."""
    v = _vectors(1)
    ffn = _ffn(264, "silu", 2)
    block = moe.MoEBlock(ffn, v[0], dropout=0.25)
    r, dr = (torch.randn(S.T, S.d, device="cuda") for _ in range(2))
    rng = torch.tensor([9, 1], device="cuda")
    out = block(r, save=True, rng=rng)
    g = block.backward(dr)
    mask = op.dropout_mask(S.T, S.d, 0.25, 9, 1)
    _, n, _, rq, _ = op.norm_residual(to_np(r), gamma_pre=to_np(v[0]))
    y, _, a = op.gated_ffn(n, to_np(ffn.W1), to_np(ffn.W2))
    r2 = op.norm_residual(to_np(r), y, mask=mask)[0]
    assert rel_l2(to_np(out.r), r2) <= 4 * 2.0 ** -8
    b = op.norm_residual_backward(r2, to_np(dr), None, y, mask=mask)
    dx, dW1, dW2 = op.gated_ffn_backward(n, a, b["dy"][0], to_np(ffn.W1), to_np(ffn.W2))
    e = op.norm_residual_backward(to_np(r), to_np(dr), dx, gamma_pre=to_np(v[0]), rstd_pre=rq)
    for got, want in ((g["dr"], e["dr"][0]), (g["dW1"], dW1), (g["dW2"], dW2), (g["dgamma_pre"], e["dgamma_pre"][0])):
        assert rel_l2(to_np(got), want) <= 4 * 2.0 ** -8


def test_step_in_a_graph():
    """A captured step of a block with a shared expert and dropout whose call number counts up in the graph."""
    layer, shared = _layer(), _ffn(136, "silu", 1)
    block = moe.MoEBlock(layer, torch.ones(S.d, device="cuda"), shared=shared, dropout=0.1)
    r, dr = (torch.randn(S.T, S.d, device="cuda") for _ in range(2))
    rng = torch.tensor([3, 0], device="cuda")

    def step():
        out = block(r, save=True, rng=rng)
        g = block.backward(dr)
        return [out.r] + [g[k] for k in ("dr", "dW1", "dW2", "dWr", "shared_dW1", "shared_dW2", "dgamma_pre")]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
        rng[1] += 1
    seen = []
    for k in range(3):
        graph.replay()
        torch.cuda.synchronize()
        seen.append([t.clone() for t in got])
    assert rng.tolist() == [3, 3] and moe.device_status() == 0
    assert not torch.equal(seen[0][0], seen[1][0])
    for k in range(3):
        rng[1] = k
        for a, b in zip(step(), seen[k]):
            assert torch.equal(a, b)


def test_a_block_keeps_one_call():
    layer, shared = _layer(), _ffn(136, "silu", 1)
    block = moe.MoEBlock(layer, torch.ones(S.d, device="cuda"), shared=shared)
    r = torch.randn(S.T, S.d, device="cuda")
    block(r, save=True)
    shared(r.to(BF16))
    with pytest.raises(RuntimeError, match="has run"):
        block.backward(r)
    with pytest.raises(ValueError, match="shared"):
        moe.MoEBlock(shared, torch.ones(S.d, device="cuda"), shared=shared)
    block = moe.MoEBlock(layer, torch.ones(S.d, device="cuda"), dropout=1.5)
    with pytest.raises(moe.MoEError, match="INVALID"):
        block(r, rng=torch.tensor([0, 0], device="cuda"))
    assert np.isfinite(to_np(block(r).r)).all()
