"""The largest sizes of the feed-forward: what its kernels cannot count in 32 bits,
or could not add up within the time that a wait lasts, is refused on the host."""
import pytest

import dropless_moe_expert_gb300 as moe

FAKE, BIG, LONG, ROWS = 1 << 20, 1 << 62, 1 << 27, (1 << 31) - 256


def _forward(T, d, f):
    """Its status, with a workspace that is too small where the sizes are taken."""
    return moe.lib.moe_gated_ffn(FAKE, FAKE, FAKE, None, 0, T, d, f, FAKE, None, FAKE, 0, None)


def _backward(T, d, f, dx=FAKE, dW1=FAKE, dW2=FAKE):
    return moe.lib.moe_gated_ffn_backward(FAKE, FAKE, FAKE, FAKE, FAKE, None, 0, T, d, f, dx, dW1, dW2, 0, FAKE, 0, None)


@pytest.mark.parametrize("size", [(ROWS, 8, 8), (1, LONG, 8), (1, 8, LONG // 2), (4096, 4096, 14336)])
def test_taken(size):
    T, d, f = size
    n = moe.lib.moe_gated_ffn_workspace_size(*size)
    assert n >= 2 * T * f and moe.lib.moe_gated_ffn_backward_workspace_size(*size) >= 3 * n
    assert _forward(*size) == 3 and _backward(*size, dW1=None, dW2=None) == 3   # the workspace, asked for last


@pytest.mark.parametrize("size", [(ROWS + 1, 8, 8), ((1 << 31) - 1, 8, 8), (1, LONG + 8, 8), (1, (1 << 31) - 8, 8),
                                  (1, 8, LONG // 2 + 8), (1, 8, (1 << 30) - 8)])
def test_refused(size):
    assert moe.lib.moe_gated_ffn_workspace_size(*size) == 0 and moe.lib.moe_gated_ffn_backward_workspace_size(*size) == 0
    assert _forward(*size) == 2 and _backward(*size) == 2 and _backward(*size, dW1=None, dW2=None) == 2


def test_sums_over_the_tokens():
    for kw in (dict(dW1=None), dict(dW2=None), dict(dx=None), {}):
        assert _backward(LONG, 8, 8, **kw) == 3 and _backward(LONG + 1, 8, 8, **kw) == 2
    assert _backward(LONG + 1, 8, 8, dW1=None, dW2=None) == 3
