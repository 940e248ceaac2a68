"""A layer's call that is refused leaves nothing behind that backward() would
take for its pre-activations.  On the host, with a library whose calls are recorded."""
import pytest
import torch

import dropless_moe_expert_gb300 as moe

from test_buffers_again import BF16, D, F, F32, Here, T, calls, here  # noqa: F401 (a fixture)


def _ffn():
    ffn = moe.GatedFFN(here(2 * F, D), here(D, F), T_max=T)
    ffn.workspace, ffn._preact_buf = here(ffn.workspace.numel(), dtype=torch.uint8), here(T, 2 * F)
    return ffn


GRADS = dict(dx=here(T, D), dW1=here(2 * F, D), dW2=here(D, F))
WORKSPACE = here(int(moe.lib.moe_gated_ffn_backward_workspace_size(T, D, F)), dtype=torch.uint8)
BAD = [dict(x=here(T, D, dtype=F32)), dict(x=here(T, 2 * D)), dict(add=here(T, 2 * D)), dict(out=here(T + 1, D)),
       dict(x=here(2 * T, D)[::2]), dict(x=here(D, T).t())]


@pytest.mark.parametrize("bad", BAD, ids=[f"{k} {tuple(v.shape)} {v.dtype}" for b in BAD for k, v in b.items()])
@pytest.mark.parametrize("before", [False, True])
def test_feed_forward(calls, bad, before):  # noqa: F811
    ffn = _ffn()
    good = dict(x=here(T, D), out=here(T, D), add=here(T, D))
    ffn(**good, save_preact=before)
    with pytest.raises((ValueError, TypeError)):
        ffn(**{**good, **bad}, save_preact=True)
    calls.clear()
    with pytest.raises(RuntimeError, match="save_preact"):
        ffn.backward(good["x"], good["x"], GRADS, WORKSPACE)
    assert not calls
    ffn(**good, save_preact=True)
    ffn.backward(good["x"], good["x"], GRADS, WORKSPACE)
    assert [n for n, _ in calls] == ["moe_gated_ffn", "moe_gated_ffn_backward"]


def test_feed_forward_that_the_library_refuses(calls, monkeypatch):  # noqa: F811
    ffn, x = _ffn(), here(T, D)
    ffn(x, out=here(T, D), save_preact=True)
    with monkeypatch.context() as m:
        m.setattr(moe, "_check", lambda code, where: (_ for _ in ()).throw(RuntimeError(where)))
        with pytest.raises(RuntimeError, match="moe_gated_ffn"):
            ffn(x, out=here(T, D), save_preact=True)
    with pytest.raises(RuntimeError, match="save_preact"):
        ffn.backward(x, x, GRADS, WORKSPACE)


def test_routed_experts(calls, monkeypatch):  # noqa: F811
    """Without pre-activations of its own the layer's backward makes them anew; it never takes what no call has written."""
    E, K = 8, 2
    layer = moe.MoELayer(here(D, E, dtype=F32), here(E, dtype=F32), here(E, 2 * F, D), here(E, D, F), K, T)
    layer._preact_buf = here(T * K * 2 * F)
    monkeypatch.setattr(moe, "_stream", lambda s=None: 0)
    x, out = here(T, D), here(T, D)
    layer(x, out=out, save_preact=True)
    with pytest.raises((ValueError, TypeError)):
        layer(here(T, D, dtype=F32), out=out, save_preact=True)
    assert layer.preact is None
    layer(x, out=out, save_preact=True)
    assert layer.preact is not None and layer.calls == 3
