"""Pins of the oracle of the operators around the layer (CPU): closed forms
and brute force for the forward values, central differences for the gradients.

Differences: with step h the truncation error is about h^2 / 6 of a third
derivative of order one and the rounding error 2^-53 |f| / h; at h = 1e-5 both
are under 1e-10 |f|, so 1e-6 of the gradient's magnitude is a wide bound."""
import itertools

import numpy as np
import pytest

from oracle import operators as op

H, TOL = 1e-5, 1e-6


def _difference(f, x):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        up, dn = x.copy(), x.copy()
        up[i] += H
        dn[i] -= H
        g[i] = (f(up) - f(dn)) / (2 * H)
    return g


def _close(value, ref, mag):
    assert np.all(np.abs(value - ref) <= TOL * (mag + 1.0))


def test_choice_by_brute_force():
    rng = np.random.default_rng(1)
    for score, groups, keep, top, bias in itertools.product(("sigmoid", "softmax"), (1, 2, 4), (1, 2), (1, 2), (0, 1)):
        if keep > groups:
            continue
        E, K = 12, 3
        L = rng.normal(size=(6, E))
        b = rng.normal(size=E) * 0.3 if bias else None
        idx, w, s = op.route_scored(L, K, score, groups, keep, top, True, 2.0, b)
        for t in range(6):
            c = s[t] + (0 if b is None else b)
            runs = [list(range(g * E // groups, (g + 1) * E // groups)) for g in range(groups)]
            best = sorted(range(groups), key=lambda g: -sum(sorted((c[e] for e in runs[g]), reverse=True)[:top]))[:keep]
            open_ = [e for g in best for e in runs[g]]
            assert idx[t].tolist() == sorted(open_, key=lambda e: -c[e])[:K]
        assert np.allclose(w.sum(axis=1), 2.0)
    assert np.allclose(op.expert_scores(L, "softmax").sum(axis=1), 1.0)


def test_valid_choice_accepts_only_what_the_errors_allow():
    c = np.array([[0.9, 0.5, 0.5 + 1e-9, 0.1, 0.3, 0.2, 0.05, 0.01]])
    err = np.full_like(c, 1e-8)

    def ok(*idx):
        return bool(op.valid_choice(np.array([idx]), c, err, len(idx))[0])

    assert ok(0, 2, 1) and ok(0, 1, 2) and ok(0, 1)       # the near tie either way
    assert not ok(0, 4) and not ok(1, 0) and not ok(0, 0) and not ok(0, 8)
    runs = lambda *idx: bool(op.valid_choice(np.array([idx]), c, err, len(idx), 2, 1, 2, np.full((1, 2), 1e-8))[0])  # noqa: E731
    assert runs(0, 2) and not runs(0, 4) and not runs(4, 5)
    idx, *_ = op.route_scored(np.log(c / (1 - c)), 2, n_group=2, topk_group=1, group_top=2)
    assert idx.tolist() == [[0, 2]]


def test_ties_go_to_the_lower_index():
    idx, w, _ = op.route_scored(np.zeros((2, 16)), 5, "sigmoid", 4, 2, 2, False, 1.0)
    assert idx.tolist() == [[0, 1, 2, 3, 4]] * 2 and np.all(w == 0.5)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_routing_gradient_is_that_of_differences(score, renorm):
    rng = np.random.default_rng(2)
    L, dw = rng.normal(size=(3, 7)), rng.normal(size=(3, 3))
    idx = np.array([[0, 3, 6], [2, 1, 5], [4, 0, 1]])
    g, mag = op.route_scored_backward(L, idx, dw, score, renorm, 1.5)
    ref = _difference(lambda x: float(np.sum(dw * op.route_scored_weights(x, idx, score, renorm, 1.5))), L)
    _close(g, ref, mag)
    assert np.all(mag >= np.abs(g) * (1 - 1e-12))


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("pre", [True, False])
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
def test_norm_gradients_are_those_of_differences(post, pre, gate):
    rng = np.random.default_rng(3)
    T, d, a, eps = 3, 6, 0.7, 0.05
    v = dict(r=rng.normal(size=(T, d)), y=rng.normal(size=(T, d)))
    if post:
        v["gamma_post"] = rng.normal(size=d)
    if pre:
        v["gamma_pre"] = rng.normal(size=d)
    if gate != "none":
        v["gate"] = rng.normal(size=d if gate == "channel" else (T, 1))
    dr, dn = rng.normal(size=(T, d)), rng.normal(size=(T, d))

    def loss(**at):
        x, n, *_ = op.norm_residual(at.pop("r"), at.pop("y"), res_scale=a, eps=eps, **at)
        return float(np.sum(dr * x) + (np.sum(dn * n) if pre else 0.0))

    x, _, rp, rq, _ = op.norm_residual(v["r"], v["y"], v.get("gamma_post"), v.get("gate"), v.get("gamma_pre"), a, eps)
    got = op.norm_residual_backward(x, dr, dn if pre else None, v["y"], v.get("gamma_post"), v.get("gate"),
                                    v.get("gamma_pre"), a, rp, rq)
    assert set(got) == {"d" + k for k in v}
    for k in v:
        value, mag = got["d" + k]
        _close(value, _difference(lambda z: loss(**{**v, k: z}), v[k]), mag)


def test_norm_of_the_stream_alone():
    rng = np.random.default_rng(4)
    r, g, dn, dr = (rng.normal(size=s) for s in ((2, 5), (5,), (2, 5), (2, 5)))
    x, n, rp, rq, _ = op.norm_residual(r, gamma_pre=g)
    assert rp is None and np.array_equal(x, r)
    assert np.allclose(np.mean((n / g) ** 2, axis=1), 1.0, atol=1e-5)
    got = op.norm_residual_backward(r, dr, dn, gamma_pre=g, rstd_pre=rq)
    _close(got["dr"][0], _difference(lambda z: float(np.sum(dr * z) + np.sum(dn * op.norm_residual(z, gamma_pre=g)[1])),
                                     r), got["dr"][1])
    assert set(got) == {"dr", "dgamma_pre"}


def test_gradient_norm():
    assert op.grad_norm([np.full(9, 2.0), np.full((4, 4), -2.0)]) == 10.0
    assert op.clip_factor(10.0, 5.0) == 5.0 / (10.0 + 1e-6) and op.clip_factor(1.0, 5.0) == 1.0
