"""The Python objects of the operators around the layer: their copies, buffers
that are replaced or used in another form, streams, and a layer that several
blocks share."""
import copy
import ctypes
import dataclasses
import gc
import pickle

import pytest
import torch

import dropless_moe_expert_gb300 as moe


# ------------------------------------------------------------------ RouteRule
def _fields(struct):
    return tuple(getattr(struct, n) for n, _ in struct._fields_)


@pytest.mark.parametrize("how", [copy.copy, copy.deepcopy, dataclasses.replace, lambda r: pickle.loads(pickle.dumps(r))],
                         ids=["copy", "deepcopy", "replace", "pickle"])
def test_copies_of_a_rule_pass_their_own_values(how):
    """What a copy hands to the library is its own struct, also when the original is gone."""
    original = moe.RouteRule("softmax", 8, 4, 2, True, 2.5)
    rule = how(original)
    assert rule == original
    del original
    gc.collect()
    others = [moe.RouteRule("sigmoid", 1, 1, 1, False, 9.0) for _ in range(64)]   # may take the freed memory
    assert rule._c == ctypes.addressof(rule._struct)
    assert _fields(moe._RouteRule.from_address(rule._c)) == (1, 8, 4, 2, 1, 2.5)
    assert len(others) == 64
