"""Operators around the layer, in fp64 -- TEST INFRASTRUCTURE ONLY.

Routing by scores, the norms with gate and residual between two layers, and
the global gradient norm, each straight from its definition (include/moe.h)
and with the gradients' formulas; it shares no code with the CUDA library.
Pins (central differences, closed forms): tests/test_oracle_operators.py.
Next to a value the gradients return its magnitude: the sum of its terms'
magnitudes, for error bounds that scale with the terms.
"""
from __future__ import annotations

import numpy as np

EPS_SUM = 1e-20


def expert_scores(L, score):
    L = np.asarray(L, np.float64)
    if score == "sigmoid":
        return 1.0 / (1.0 + np.exp(-L))
    z = np.exp(L - L.max(axis=1, keepdims=True))
    return z / z.sum(axis=1, keepdims=True)


def _ranked(c):
    """Indices by descending value, the lower index first on ties."""
    return np.argsort(-c, axis=-1, kind="stable")


def route_scored(L, K, score="sigmoid", n_group=1, topk_group=1, group_top=1, renorm=True, scale=1.0, sel_bias=None):
    """idx [T, K], w [T, K] and the scores s [T, E]."""
    s = expert_scores(L, score)
    T, E = s.shape
    per = E // n_group
    c = s if sel_bias is None else s + np.asarray(sel_bias, np.float64)
    open_ = np.ones((T, n_group), bool)
    if topk_group < n_group:
        g = run_scores(c, n_group, group_top)
        open_ = np.zeros((T, n_group), bool)
        np.put_along_axis(open_, _ranked(g)[:, :topk_group], True, axis=1)
    closed = ~np.repeat(open_, per, axis=1)
    # closed runs rank below everything, whatever their values
    idx = np.lexsort((np.broadcast_to(np.arange(E), c.shape), -c, closed), axis=1)[:, :K]
    t = np.take_along_axis(s, idx, axis=1)
    w = scale * t / (t.sum(axis=1, keepdims=True) + EPS_SUM) if renorm else scale * t
    return idx.astype(np.int32), w, s


def run_scores(c, n_group, group_top):
    T, E = c.shape
    per = E // n_group
    return -np.sort(-c.reshape(T, n_group, per), axis=2)[:, :, :min(group_top, per)].sum(axis=2)


def valid_choice(idx, c, err, K, n_group=1, topk_group=1, group_top=1, gerr=None):
    """Per token, whether `idx` is a choice that some values within `err` of c
    (and run scores within `gerr` of theirs) would give: distinct experts, none
    in a run that is surely closed, in descending order within the errors, and
    none passed over, in a run that is surely open, that is surely larger."""
    T, E = c.shape
    per = E // n_group
    lo, hi = c - err, c + err
    sure_open = np.ones((T, n_group), bool)
    sure_closed = np.zeros((T, n_group), bool)
    if topk_group < n_group:
        g = run_scores(c, n_group, group_top)
        glo, ghi = g - gerr, g + gerr
        above = (ghi[:, None, :] >= glo[:, :, None]).sum(axis=2) - 1     # others that may be at least as large
        sure_open = above < topk_group
        sure_closed = (glo[:, None, :] > ghi[:, :, None]).sum(axis=2) >= topk_group
    idx = np.asarray(idx, np.int64)
    ok = (np.sort(idx, axis=1)[:, 1:] != np.sort(idx, axis=1)[:, :-1]).all(axis=1) & (idx >= 0).all(1) & (idx < E).all(1)
    idx = np.clip(idx, 0, E - 1)
    ok &= ~np.take_along_axis(np.repeat(sure_closed, per, axis=1), idx, axis=1).any(axis=1)
    h, low = np.take_along_axis(hi, idx, axis=1), np.take_along_axis(lo, idx, axis=1)
    ok &= (h[:, :-1] >= low[:, 1:]).all(axis=1)
    rest = np.repeat(sure_open, per, axis=1)
    np.put_along_axis(rest, idx, False, axis=1)
    return ok & (np.where(rest, lo, -np.inf).max(axis=1) <= h.min(axis=1))


def route_scored_weights(L, idx, score="sigmoid", renorm=True, scale=1.0):
    """The weights of a given choice."""
    t = np.take_along_axis(expert_scores(L, score), np.asarray(idx, np.int64), axis=1)
    return scale * t / (t.sum(axis=1, keepdims=True) + EPS_SUM) if renorm else scale * t


def route_scored_backward(L, idx, dw, score="sigmoid", renorm=True, scale=1.0):
    """dL [T, E] of sum(dw * w) for a given choice, and its magnitudes."""
    s = expert_scores(L, score)
    idx = np.asarray(idx, np.int64)
    dw = np.asarray(dw, np.float64)
    t = np.take_along_axis(s, idx, axis=1)
    if renorm:
        S = t.sum(axis=1, keepdims=True) + EPS_SUM
        ds = scale * (dw - np.sum(dw * t / S, axis=1, keepdims=True)) / S
        mag = abs(scale) * (np.abs(dw) + np.sum(np.abs(dw) * t / S, axis=1, keepdims=True)) / S
    else:
        ds, mag = scale * dw, abs(scale) * np.abs(dw)
    full, fmag = np.zeros_like(s), np.zeros_like(s)
    np.put_along_axis(full, idx, ds, axis=1)
    np.put_along_axis(fmag, idx, mag, axis=1)
    if score == "sigmoid":
        slope = s * (1.0 / (1.0 + np.exp(np.asarray(L, np.float64))))
        return full * slope, fmag * slope
    return (s * (full - np.sum(s * full, axis=1, keepdims=True)),
            s * (fmag + np.sum(s * fmag, axis=1, keepdims=True)))


def norm_residual(r, y=None, gamma_post=None, gate=None, gamma_pre=None, res_scale=1.0, eps=1e-6):
    """r', n, rstd_post, rstd_pre, and |res_scale r| + |gate u|."""
    x = np.asarray(r, np.float64)
    mag = np.abs(x)
    rp = rq = n = None
    if y is not None:
        u = np.asarray(y, np.float64)
        if gamma_post is not None:
            rp = 1.0 / np.sqrt(np.mean(u * u, axis=1) + eps)
            u = u * rp[:, None] * np.asarray(gamma_post, np.float64)
        if gate is not None:
            u = u * np.asarray(gate, np.float64)
        mag = np.abs(res_scale * x) + np.abs(u)
        x = res_scale * x + u
    if gamma_pre is not None:
        rq = 1.0 / np.sqrt(np.mean(x * x, axis=1) + eps)
        n = x * rq[:, None] * np.asarray(gamma_pre, np.float64)
    return x, n, rp, rq, mag


def norm_residual_backward(r_out, dr_out, dn=None, y=None, gamma_post=None, gate=None, gamma_pre=None, res_scale=1.0,
                           rstd_post=None, rstd_pre=None):
    """Gradients for dr_out and dn with the rows' factors given; a dict of
    (value, magnitude) for dr, dy, dgamma_pre, dgamma_post, dgate."""
    x = np.asarray(r_out, np.float64)
    D = np.zeros_like(x) if dr_out is None else np.asarray(dr_out, np.float64)
    Dm = np.abs(D)
    out = {}
    if gamma_pre is not None:
        f = np.asarray(rstd_pre, np.float64)[:, None]
        dn = np.asarray(dn, np.float64)
        h = dn * np.asarray(gamma_pre, np.float64)
        out["dgamma_pre"] = ((dn * x * f).sum(axis=0), np.abs(dn * x * f).sum(axis=0))
        D = D + f * (h - x * f * f * np.mean(h * x, axis=1, keepdims=True))
        Dm = Dm + f * (np.abs(h) + np.abs(x) * f * f * np.mean(np.abs(h * x), axis=1, keepdims=True))
    a = 1.0 if y is None else res_scale
    out["dr"] = (a * D, abs(a) * Dm)
    if y is None:
        return out
    y = np.asarray(y, np.float64)
    v = y if gamma_post is None else y * np.asarray(rstd_post, np.float64)[:, None]
    w = 1.0 if gamma_post is None else np.asarray(gamma_post, np.float64)
    k, km = D, Dm
    if gate is not None:
        g = np.asarray(gate, np.float64)
        axis, keep = ((0, False) if g.ndim == 1 else (1, True))
        out["dgate"] = ((v * w * D).sum(axis=axis, keepdims=keep), (np.abs(v * w) * Dm).sum(axis=axis, keepdims=keep))
        k, km = k * g, km * np.abs(g)
    if gamma_post is not None:
        f = np.asarray(rstd_post, np.float64)[:, None]
        out["dgamma_post"] = ((k * v).sum(axis=0), (km * np.abs(v)).sum(axis=0))
        k, km = k * w, km * np.abs(w)
        km = f * (km + np.abs(y) * f * f * np.mean(km * np.abs(y), axis=1, keepdims=True))
        k = f * (k - y * f * f * np.mean(k * y, axis=1, keepdims=True))
    out["dy"] = (k, km)
    return out


def grad_norm(grads):
    return float(np.sqrt(sum(float(np.sum(np.square(np.asarray(g, np.float64)))) for g in grads)))


def clip_factor(norm, max_norm):
    return min(1.0, max_norm / (norm + 1e-6))
