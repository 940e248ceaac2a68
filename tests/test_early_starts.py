"""Kernels that start before the one in front of them has ended, on what that one
wrote by plain stores and these read by bulk or tensor copies: the same bits as
with a synchronize between the calls."""
import pytest
import torch

import dropless_moe_expert_gb300 as moe

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def _normal(*shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return scale * torch.randn(*shape, generator=g, device="cuda")


def _weights(d, f, seed):
    return _normal(2 * f, d, seed=seed, scale=d ** -0.5).to(BF16), _normal(d, f, seed=seed + 1, scale=f ** -0.5).to(BF16)


def _bits(step, n=20):
    """step(between) calls between() after each of its calls: nothing, or a synchronize."""
    want = [t.clone() for t in step(torch.cuda.synchronize)]
    torch.cuda.synchronize()
    for _ in range(n):
        for a, b in zip(step(lambda: None), want):
            assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(lambda: None)
    for _ in range(n):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert moe.device_status() == 0


# T, d, f: both layers without tiles, with K shared, either behind the other, and CTA pairs behind both
@pytest.mark.parametrize("T,d,f", [(1, 1024, 512), (48, 4096, 1536), (64, 512, 4096), (100, 1416, 520), (129, 328, 776),
                                   (300, 1024, 2048), (700, 512, 640)])
def test_feed_forwards_in_a_row(T, d, f):
    """y of one layer is x of the next; and back, where dx of one is dy of the other."""
    x, dy = _normal(T, d, seed=0).to(BF16), _normal(T, d, seed=1).to(BF16)
    layers = [moe.GatedFFN(*_weights(d, n, seed), act, T_max=T)
              for n, act, seed in ((f, "silu", 2), (f, "gelu", 4), (f + 128, "gelu_tanh", 6))]

    def step(between):
        xs, g = [x], dy
        for layer in layers:
            xs.append(layer(xs[-1], save_preact=True))
            between()
        out = [*xs[1:]]
        for layer, a in zip(reversed(layers), reversed(xs[:-1])):
            d_ = layer.backward(a, g)
            between()
            g = d_["dx"]
            out += [g, d_["dW1"], d_["dW2"]]
        return out

    _bits(step)


@pytest.mark.parametrize("dt", [torch.float32, BF16])
@pytest.mark.parametrize("T,d,f", [(1, 1024, 512), (16, 4096, 512), (48, 2048, 768), (129, 2624, 776), (700, 512, 640)])
def test_norms_between_feed_forwards(T, d, f, dt):
    """Norms read by bulk copies what a layer, or the norm before them, has just written, and the other way round."""
    r0, dr = _normal(T, d, seed=0).to(dt), _normal(T, d, seed=1).to(dt)
    gammas = [1 + _normal(d, seed=10 + k, scale=0.1) for k in range(3)]
    layers = [moe.GatedFFN(*_weights(d, f, 2 * k), T_max=T) for k in range(2)]
    rng = torch.tensor([4, 2], device="cuda")

    def step(between):
        def do(call, *a, **kw):
            out = call(*a, **kw)
            between()
            return out

        n = do(moe.norm_residual, r0, gamma_pre=gammas[0])
        rows, out = [], []
        for k, layer in enumerate(layers):
            y = do(layer, n.n, save_preact=True)
            drop = dict(dropout=0.2, rng=rng) if k else {}
            m = do(moe.norm_residual, n.r, y, gamma_post=gammas[1], gamma_pre=gammas[k + 1], **drop)
            rows.append((n, y, m, drop))
            out += [y, m.r, m.n]
            n = m
        g, dn = dr, n.n
        for k in (1, 0):
            n, y, m, drop = rows[k]
            h = do(moe.norm_residual_backward, m.r, g, dn, y, gamma_post=gammas[1], gamma_pre=gammas[k + 1],
                   rstd_post=m.rstd_post, rstd_pre=m.rstd_pre, **drop)
            w = do(layers[k].backward, n.n, h.dy)
            g, dn = h.dr, w["dx"]
            out += [h.dr, h.dy, h.dgamma_pre, h.dgamma_post, w["dx"], w["dW1"], w["dW2"]]
        return out

    _bits(step)


@pytest.mark.parametrize("T,d,f", [(1, 1024, 512), (48, 4096, 1536), (100, 1416, 520), (129, 328, 776), (200, 256, 8192)])
def test_weights_made_just_before(T, d, f):
    """Weights that a plain kernel has stored right before the call: the second and the third kernel of it ask
    for theirs before the ones in front of them have ended."""
    x, dy = _normal(T, d, seed=0).to(BF16), _normal(T, d, seed=1).to(BF16)
    made = [_weights(d, f, 2 * k) for k in range(3)]
    W1, W2 = (torch.empty_like(t) for t in made[0])
    ffn, pre = moe.GatedFFN(W1, W2, T_max=T), torch.empty(T, 2 * f, dtype=BF16, device="cuda")
    one = torch.ones((), dtype=BF16, device="cuda")

    def step(between):
        out = []
        for a, b in made:
            torch.mul(a, one, out=W1)
            torch.mul(b, one, out=W2)
            between()
            y = ffn(x, save_preact=True)
            between()
            pre.copy_(ffn.preact)
            torch.mul(b, one, out=W2)
            torch.mul(a, one, out=W1)
            between()
            g = moe.gated_ffn_backward(x, pre, dy, W1, W2)
            between()
            out += [y, g.dx, g.dW1, g.dW2]
        return out

    _bits(step)
