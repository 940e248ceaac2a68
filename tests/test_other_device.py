"""The feed-forward and the norms with dropout work on the current device: a
tensor of another one is refused wherever it stands, before anything is
launched.  On the host, with tensors that say where they are."""
import pytest
import torch

import dropless_moe_expert_gb300 as moe

from test_buffers_again import BF16, D, F, F32, Here, T, calls, here  # noqa: F401 (a fixture)


class There(Here):
    """One of the second device."""

    def get_device(self):
        return 1


def _each_elsewhere(calls, run, args):
    """run(**args) is made; with any one of the tensors on another device it is refused."""
    run(**args)
    assert len(calls) == 1
    for name, t in args.items():
        calls.clear()
        with pytest.raises(ValueError, match="device 1"):
            run(**{**args, name: t.as_subclass(There)})
        assert not calls, name


def test_feed_forward(calls):  # noqa: F811
    n = int(moe.lib.moe_gated_ffn_workspace_size(T, D, F))
    args = dict(x=here(T, D), W1=here(2 * F, D), W2=here(D, F), add=here(T, D), out=here(T, D), preact=here(T, 2 * F),
                workspace=here(n, dtype=torch.uint8))
    _each_elsewhere(calls, moe.gated_ffn, args)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_feed_forward_backward(calls, dtype):  # noqa: F811
    n = int(moe.lib.moe_gated_ffn_backward_workspace_size(T, D, F))
    args = dict(x=here(T, D), preact=here(T, 2 * F), dy=here(T, D), W1=here(2 * F, D), W2=here(D, F), add=here(T, D),
                dx=here(T, D), dW1=here(2 * F, D, dtype=dtype), dW2=here(D, F, dtype=dtype), workspace=here(n, dtype=torch.uint8))

    def run(dx, dW1, dW2, workspace, **kw):
        return moe.gated_ffn_backward(**kw, out=moe.GatedFFNGrads(dx, dW1, dW2, workspace))
    _each_elsewhere(calls, run, args)


def _object():
    ffn = moe.GatedFFN(here(2 * F, D), here(D, F), T_max=T)
    ffn.workspace, ffn._preact_buf = here(ffn.workspace.numel(), dtype=torch.uint8), here(T, 2 * F)
    return ffn


def test_feed_forward_object(calls):  # noqa: F811
    ffn = _object()
    _each_elsewhere(calls, ffn, dict(x=here(T, D), add=here(T, D), out=here(T, D)))
    for name in ("W1", "W2", "workspace", "_preact_buf"):
        ffn = _object()
        x, out = here(T, D), here(T, D)
        ffn(x, out=out, save_preact=True)
        setattr(ffn, name, getattr(ffn, name).clone().as_subclass(There))
        calls.clear()
        with pytest.raises(ValueError, match="device 1"):
            ffn(x, out=out, save_preact=True)
        assert not calls


def test_objects_of_the_device_that_was_current(calls, monkeypatch):  # noqa: F811
    """The current device changes between two calls: what was accepted on the first one is not on the second."""
    ffn, x = _object(), here(T, D)
    ws = here(int(moe.lib.moe_gated_ffn_backward_workspace_size(T, D, F)), dtype=torch.uint8)
    grads = moe.GatedFFNGrads(here(T, D), here(2 * F, D), here(D, F), ws)
    rng, r, y = here(2, dtype=torch.int64), here(T, D, dtype=F32), here(T, D)
    out = moe.NormResidual(here(T, D, dtype=F32), rng=here(2, dtype=torch.int64))
    rows = moe.NormResidualGrads(here(T, D, dtype=F32), here(T, D),
                                 workspace=here(int(moe.lib.moe_norm_residual_backward_workspace_size(T, D)), dtype=torch.uint8))

    def runs(k):
        def on(t):
            return t.as_subclass(k)
        return [lambda: ffn(on(x), out=on(y)),
                lambda: moe.gated_ffn_backward(on(x), on(here(T, 2 * F)), on(x), on(here(2 * F, D)), on(here(D, F)), out=grads),
                lambda: moe.norm_residual(on(r), on(y), dropout=0.1, rng=on(rng), out=out),
                lambda: moe.norm_residual_backward(on(r), on(r), None, on(y), dropout=0.1, rng=on(rng), out=rows)]
    for run in runs(Here):
        run()
    assert len(calls) == 4
    calls.clear()
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    for run in runs(There):
        with pytest.raises(ValueError, match="device 0"):
            run()
    assert not calls


def test_dropout(calls):  # noqa: F811
    f32 = dict(dtype=F32)
    args = dict(r=here(T, D, **f32), y=here(T, D), gamma_post=here(D, **f32), gate=here(D, **f32), gamma_pre=here(D, **f32),
                rng=here(2, dtype=torch.int64))
    outs = dict(o_r=here(T, D, **f32), o_n=here(T, D), o_post=here(T, **f32), o_pre=here(T, **f32),
                o_rng=here(2, dtype=torch.int64))

    def run(o_r, o_n, o_post, o_pre, o_rng, **kw):
        return moe.norm_residual(**kw, dropout=0.1, out=moe.NormResidual(o_r, o_n, o_post, o_pre, o_rng))
    _each_elsewhere(calls, run, {**args, **outs})
    grads = dict(o_dr=here(T, D, **f32), o_dy=here(T, D), o_gq=here(D, **f32), o_gp=here(D, **f32), o_g=here(D, **f32),
                 o_ws=here(int(moe.lib.moe_norm_residual_backward_workspace_size(T, D)), dtype=torch.uint8))
    more = dict(dr=here(T, D, **f32), dn=here(T, D), rstd_post=here(T, **f32), rstd_pre=here(T, **f32))

    def back(o_dr, o_dy, o_gq, o_gp, o_g, o_ws, **kw):
        return moe.norm_residual_backward(**kw, dropout=0.1, out=moe.NormResidualGrads(o_dr, o_dy, o_gq, o_gp, o_g, o_ws))
    calls.clear()
    _each_elsewhere(calls, back, {**args, **more, **grads})
    with pytest.raises(ValueError, match="device 1"):
        moe.norm_residual(args["r"], args["y"], dropout=0.1, rng=args["rng"].as_subclass(There))
    with pytest.raises(ValueError, match="device 1"):
        moe.norm_residual_backward(args["r"], more["dr"], None, args["y"], dropout=0.1, rng=args["rng"].as_subclass(There))
