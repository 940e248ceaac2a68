"""The dropout's state and where a call leaves it: the same two words or apart.
Refused on the host, before anything is launched."""
import pytest

import dropless_moe_expert_gb300 as moe

FAKE = 1 << 20   # a 16-byte aligned address; never dereferenced


@pytest.mark.parametrize("rng,rng_out", [(FAKE, FAKE + 8), (FAKE + 8, FAKE)])
def test_half_of_the_state_is_not_written_over(rng, rng_out):
    """One word of it would be written while other rows still read it."""
    before = moe.launch_count()
    args = [FAKE, 0, FAKE, None, None, 0, 1.0, None, 1e-6, 0.1, rng, 4, 128, FAKE, None, None, None, rng_out, None]
    assert moe.lib.moe_norm_residual_dropout(*args) == 1
    assert moe.launch_count() == before
