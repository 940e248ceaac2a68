"""Pins of the fp64 oracle of the gated feed-forward and of the dropout: known
answers of the generator, torch's activations, central differences."""
import numpy as np
import pytest
import torch

from oracle import operators as op

ACTS = ("silu", "gelu", "gelu_tanh", "relu")


def test_philox_known_answers():
    """The test vectors published with the generator: zeros, ones, and digits of pi."""
    assert op.philox4x32_10(0, 0, [0]) == [[0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]]
    ones = (1 << 64) - 1
    assert op.philox4x32_10(ones, ones, [ones]) == [[0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd]]
    assert op.philox4x32_10(0x299f31d0a4093822, 0x0370734413198a2e, [0x85a308d3243f6a88]) == \
        [[0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1]]


def test_dropout_mask():
    """Elements go by their 16-bit draws; rows do not depend on which are asked for; calls and seeds differ."""
    T, d, p = 37, 64, 0.25
    m = op.dropout_mask(T, d, p, 5, 9)
    w = op.philox4x32_10(5, 9, [3 * 8 + 2])[0]
    draws = [w[0] & 0xffff, w[0] >> 16, w[1] & 0xffff, w[1] >> 16, w[2] & 0xffff, w[2] >> 16, w[3] & 0xffff, w[3] >> 16]
    assert np.array_equal(m[3, 16:24] > 0, [v >= 16384 for v in draws])
    assert set(np.unique(m)) == {0.0, 1 / 0.75}
    assert np.array_equal(op.dropout_mask(T, d, p, 5, 9, rows=[3, 36]), m[[3, 36]])
    assert not np.array_equal(op.dropout_mask(T, d, p, 5, 10), m) and not np.array_equal(op.dropout_mask(T, d, p, 6, 9), m)
    # 2368 draws: six standard deviations
    assert abs((m > 0).mean() - 0.75) < 6 * np.sqrt(0.75 * 0.25 / m.size)
    assert (op.dropout_mask(T, d, 0.0, 5, 9) == 1).all()


@pytest.mark.parametrize("act", ACTS)
def test_activations(act):
    g = np.concatenate([np.linspace(-12, 12, 241), [-40.0, 40.0, 0.0]])
    t = torch.from_numpy(g).requires_grad_(True)
    f = {"silu": torch.nn.functional.silu, "relu": torch.relu, "gelu": torch.nn.functional.gelu,
         "gelu_tanh": lambda z: torch.nn.functional.gelu(z, approximate="tanh")}[act]
    y = f(t)
    y.sum().backward()
    v, slope = op.activation(act, g)
    assert np.allclose(v, y.detach().numpy(), rtol=1e-9, atol=1e-13)
    assert np.allclose(slope, t.grad.numpy(), rtol=1e-9, atol=1e-13)


@pytest.mark.parametrize("act", ACTS)
def test_feed_forward_gradients_against_differences(act):
    rng = np.random.default_rng(3)
    T, d, f = 5, 6, 7
    x, W1, W2 = rng.normal(size=(T, d)), rng.normal(size=(2 * f, d)), rng.normal(size=(d, f))
    dy, add = rng.normal(size=(T, d)), rng.normal(size=(T, d))
    y, h, a = op.gated_ffn(x, W1, W2, act, add)
    assert np.allclose(y - add, h @ W2.T) and np.allclose(a, np.einsum("td,fd->tf", x, W1))
    if act == "relu":
        assert np.abs(a[:, :f]).min() > 1e-3    # no kink within the steps
    dx, dW1, dW2 = op.gated_ffn_backward(x, a, dy, W1, W2, act)
    assert np.allclose(op.gated_ffn_backward(x, a, dy, W1, W2, act, add)[0], dx + add)
    step = 1e-5
    for at, grad in ((0, dx), (1, dW1), (2, dW2)):
        for i in rng.choice(grad.size, 12, replace=False):
            lo, hi = [x, W1, W2], [x, W1, W2]
            for side, s in ((lo, -step), (hi, step)):
                side[at] = side[at].copy()
                side[at].flat[i] += s
            diff = ((op.gated_ffn(*hi, act)[0] - op.gated_ffn(*lo, act)[0]) * dy).sum() / (2 * step)
            assert abs(diff - grad.flat[i]) <= 1e-6 * (1 + abs(diff))


@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("post", [False, True])
def test_dropout_gradients_against_differences(gate, post):
    """Of sum(dr * r') + sum(dn * n), with the same mask in both directions."""
    rng = np.random.default_rng(4)
    T, d = 6, 16
    mask = op.dropout_mask(T, d, 0.3, 11, 2)
    assert 0 < (mask == 0).sum() < mask.size
    ins = dict(r=rng.normal(size=(T, d)), y=rng.normal(size=(T, d)), gamma_pre=1 + 0.1 * rng.normal(size=d))
    if post:
        ins["gamma_post"] = 1 + 0.1 * rng.normal(size=d)
    if gate != "none":
        ins["gate"] = rng.normal(size=d if gate == "channel" else (T, 1))
    dr, dn = rng.normal(size=(T, d)), rng.normal(size=(T, d))

    def loss(v):
        r2, n, _, _, _ = op.norm_residual(res_scale=0.7, mask=mask, **v)
        return (dr * r2).sum() + (dn * n).sum()

    r2, _, rp, rq, _ = op.norm_residual(res_scale=0.7, mask=mask, **ins)
    rest = {k: v for k, v in ins.items() if k != "r"}
    g = op.norm_residual_backward(r2, dr, dn, res_scale=0.7, rstd_post=rp, rstd_pre=rq, mask=mask, **rest)
    if not post:
        assert (g["dy"][0][mask == 0] == 0).all()
    for name, key in (("r", "dr"), ("y", "dy"), ("gamma_pre", "dgamma_pre"), ("gamma_post", "dgamma_post"),
                      ("gate", "dgate")):
        if name not in ins:
            assert key not in g
            continue
        value, mag = g[key]
        assert np.all(np.abs(value) <= mag * (1 + 1e-12))
        for i in rng.choice(value.size, min(12, value.size), replace=False):
            sides = []
            for s in (-1e-5, 1e-5):
                v = {k: t.copy() for k, t in ins.items()}
                v[name].flat[i] += s
                sides.append(loss(v))
            assert abs((sides[1] - sides[0]) / 2e-5 - value.flat[i]) <= 1e-6 * (1 + abs(value.flat[i]))
