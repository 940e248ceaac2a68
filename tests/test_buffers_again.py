"""Buffers and weights that were accepted once and then replaced by another view
of the same memory: checked again, so that no call goes by an address alone.
On the host: tensors that say they are on a GPU, and a library whose calls are
recorded."""
import pytest
import torch

import dropless_moe_expert_gb300 as moe

BF16, F32 = torch.bfloat16, torch.float32


class Here(torch.Tensor):
    """A host tensor that passes for one of the current device."""
    is_cuda = property(lambda self: True)

    def get_device(self):
        return 0


def here(*shape, dtype=BF16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(Here)


@pytest.fixture
def calls(monkeypatch):
    made = []

    class Recorder:
        def __getattr__(self, name):
            if name.endswith("_size"):
                return getattr(real, name)
            return lambda *a: made.append((name, a)) or 0

    real = moe.lib
    monkeypatch.setattr(moe, "lib", Recorder())
    monkeypatch.setattr(moe, "_stream_of", lambda t, stream=None: 0)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    return made


T, D, F = 8, 64, 64


def _refused(calls, run, change, kind, match):
    """run() works, is refused after change(), and works again after what that returns."""
    run()
    calls.clear()
    back = change()
    with pytest.raises(kind, match=match):
        run()
    assert not calls
    back()
    run()
    assert len(calls) == 1


def _swap(obj, name, new):
    def change():
        old = getattr(obj, name)
        setattr(obj, name, new(old))
        assert getattr(obj, name).data_ptr() == old.data_ptr()
        return lambda: setattr(obj, name, old)
    return change


def _in_place(obj, name, new):
    def change():
        t = getattr(obj, name)
        old = t.data
        t.data = new(old)
        assert t.data_ptr() == old.data_ptr()

        def back():
            t.data = old
        return back
    return change


def _ffn():
    ffn = moe.GatedFFN(here(2 * F, D), here(D, F), T_max=T)
    ffn.workspace = here(ffn.workspace.numel(), dtype=torch.uint8)
    return ffn


VIEWS = [(lambda t: t.t(), ValueError, "contiguous"), (lambda t: t.view(torch.float16), TypeError, "must be"),
         (lambda t: t[:t.shape[0] // 2], ValueError, "shape"), (lambda t: t.view(-1), ValueError, "shape")]


@pytest.mark.parametrize("how", [_swap, _in_place])
@pytest.mark.parametrize("view", range(len(VIEWS)))
@pytest.mark.parametrize("name", ["W2", "W1"])
def test_weights_of_a_feed_forward(calls, name, view, how):
    new, kind, match = VIEWS[view]
    if name == "W1" and view == 0:
        match = "shape"
    ffn, x = _ffn(), here(T, D)
    _refused(calls, lambda: ffn(x, out=here(T, D)), how(ffn, name, new), kind, name + " must" if match == "must be" else match)


def test_workspace_of_a_feed_forward(calls):
    ffn, x = _ffn(), here(T, D)
    _refused(calls, lambda: ffn(x, out=here(T, D)), _swap(ffn, "workspace", lambda t: t.view(torch.int8)), TypeError, "workspace")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("name,new,kind,match", [
    ("dW2", lambda t: t.t(), ValueError, "dW2"), ("dW2", lambda t: t[:32], ValueError, "dW2"),
    ("dW1", lambda t: t[:32], ValueError, "dW1"), ("dx", lambda t: t[:3], ValueError, "dx"),
    ("dx", lambda t: t.view(torch.float16), TypeError, "dx"), ("dW1", lambda t: t.view(torch.int16), (TypeError, ValueError), "dW1"),
    ("workspace", lambda t: t.view(torch.int8), TypeError, "workspace")])
def test_gradients_of_a_feed_forward(calls, name, new, kind, match, dtype):
    W1, W2, x, pre = here(2 * F, D), here(D, F), here(T, D), here(T, 2 * F)
    ws = here(int(moe.lib.moe_gated_ffn_backward_workspace_size(T, D, F)), dtype=torch.uint8)
    out = moe.GatedFFNGrads(here(T, D), here(2 * F, D, dtype=dtype), here(D, F, dtype=dtype), ws)
    for how in (_swap, _in_place):
        _refused(calls, lambda: moe.gated_ffn_backward(x, pre, x, W1, W2, out=out), how(out, name, new), kind, match)


def _norm_call(out, **dropout):
    r, y, g = here(T, D, dtype=F32), here(T, D), here(D, dtype=F32)
    return lambda: moe.norm_residual(r, y, gamma_post=g, gamma_pre=g, out=out, **dropout)


@pytest.mark.parametrize("name,new,kind", [
    ("r", lambda t: t.view(torch.int32), TypeError), ("r", lambda t: t[:3], ValueError), ("n", lambda t: t[:3], ValueError),
    ("n", lambda t: t.view(D, T).t(), ValueError), ("rstd_pre", lambda t: t[:3], ValueError),
    ("rstd_post", lambda t: t.view(T, 1), ValueError), ("rng", lambda t: t.view(torch.float64), TypeError)])
def test_outputs_of_the_norms(calls, name, new, kind):
    out = moe.NormResidual(here(T, D, dtype=F32), here(T, D), here(T, dtype=F32), here(T, dtype=F32), here(2, dtype=torch.int64))
    state = here(2, dtype=torch.int64)
    for how in (_swap, _in_place):
        _refused(calls, _norm_call(out, dropout=0.1, rng=state), how(out, name, new), kind, "out." + name)
        if name != "rng":
            _refused(calls, _norm_call(out), how(out, name, new), kind, "out." + name)


@pytest.mark.parametrize("new,kind", [(lambda t: t.view(torch.float64), TypeError), (lambda t: t[::2], ValueError),
                                      (lambda t: t.view(torch.int32)[:2], TypeError)])
def test_dropout_state(calls, new, kind):
    r, y = here(T, D, dtype=F32), here(T, D)
    ws = here(int(moe.lib.moe_norm_residual_backward_workspace_size(T, D)), dtype=torch.uint8)
    out = moe.NormResidual(here(T, D, dtype=F32), rng=here(2, dtype=torch.int64))
    grads = moe.NormResidualGrads(here(T, D, dtype=F32), here(T, D), workspace=ws)
    big = here(4, dtype=torch.int64)
    for run in (lambda: moe.norm_residual(r, y, dropout=0.1, rng=state[0], out=out),
                lambda: moe.norm_residual_backward(r, r, None, y, dropout=0.1, rng=state[0], out=grads)):
        state = [big[:2]]

        def change():
            state[0] = new(big if kind is ValueError else big[:2])
            if kind is ValueError:      # [2], every other word
                assert tuple(state[0].shape) == (2,) and not state[0].is_contiguous()
            assert state[0].data_ptr() == big.data_ptr()
            return lambda: state.__setitem__(0, big[:2])
        _refused(calls, run, change, kind, "rng")


@pytest.mark.parametrize("name,new,kind", [
    ("dr", lambda t: t[:3], ValueError), ("dy", lambda t: t[:3], ValueError), ("dy", lambda t: t.view(torch.float16), TypeError),
    ("dgamma_pre", lambda t: t[:8], ValueError), ("dgamma_post", lambda t: t.view(torch.int32), TypeError),
    ("dgate", lambda t: t.view(1, T), ValueError), ("workspace", lambda t: t.view(torch.int8), TypeError)])
def test_gradients_of_the_norms(calls, name, new, kind):
    r, y, g = here(T, D, dtype=F32), here(T, D), here(D, dtype=F32)
    ws = here(int(moe.lib.moe_norm_residual_backward_workspace_size(T, D)), dtype=torch.uint8)
    out = moe.NormResidualGrads(here(T, D, dtype=F32), here(T, D), here(D, dtype=F32), here(D, dtype=F32),
                                here(T, 1, dtype=F32), ws)
    rows = here(T, dtype=F32)

    def run():
        moe.norm_residual_backward(r, r, y, y, gamma_post=g, gate=here(T, 1, dtype=F32), gamma_pre=g, rstd_post=rows,
                                   rstd_pre=rows, out=out)
    for how in (_swap, _in_place):
        _refused(calls, run, how(out, name, new), kind, "out." + name)


@pytest.mark.parametrize("name,new,kind", [
    ("topk_idx", lambda t: t[:3], ValueError), ("topk_w", lambda t: t.view(torch.int32), TypeError),
    ("counts", lambda t: t[:3], ValueError), ("row_of", lambda t: t.view(2, T).t(), ValueError),
    ("src_tok", lambda t: t[:3], ValueError), ("offsets", lambda t: t[:3], ValueError)])
def test_routing_buffers(calls, monkeypatch, name, new, kind):
    empty = torch.empty
    with monkeypatch.context() as m:
        m.setattr(torch, "empty", lambda *a, **kw: empty(*a, **kw).as_subclass(Here))
        buffers = moe.RouteBuffers(T, 16, 2, "cpu")
    logits, rule = here(T, 16, dtype=F32), moe.RouteRule()
    for how in (_swap, _in_place):
        _refused(calls, lambda: moe.route_scored(logits, 2, rule, buffers=buffers), how(buffers.routing, name, new), kind, name)


def test_nothing_is_checked_twice(calls, monkeypatch):
    """The same tensors again, another object for the same memory among them."""
    ffn, x, out = _ffn(), here(T, D), here(T, D)
    ffn(x, out=out)
    asked, check = [], moe._in
    monkeypatch.setattr(moe, "_in", lambda t, dtype, shape, name: asked.append(name) or check(t, dtype, shape, name))
    ffn.W2 = ffn.W2.view(D, F)
    ffn(x, out=out)
    assert "x" in asked and not {"W1", "W2", "workspace"} & set(asked) and len(calls) == 2


def test_in_other_modes_of_torch(calls):
    """Checks that were made in one mode hold, or are made again, in another."""
    ffn, x, out = _ffn(), here(T, D), here(T, D)
    for mode in (torch.no_grad, torch.inference_mode, torch.enable_grad, torch.inference_mode):
        with mode():
            for _ in range(2):
                ffn(x, out=out)
    ffn.W2 = torch.nn.Parameter(ffn.W2, requires_grad=False)
    assert len(calls) == 8
    with pytest.raises(ValueError, match="W2"), torch.inference_mode():
        ffn.W2 = here(D, F).t()
        ffn(x, out=out)
    assert len(calls) == 8
