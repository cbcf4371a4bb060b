"""Refusals of the bounded waits' hook, on the host."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def stree():
    from hybrid_packed_tree_b200.build import build
    build()
    from hybrid_packed_tree_b200 import stree
    return stree


def test_hook_refuses_what_it_does_not_know(stree):
    assert stree._lib.stree_set_wait_hook(None) == 1
    for bad in (dict(fault=2), dict(fault=-1), dict(wait_ns=4_000_000_001)):
        with pytest.raises(stree.StreeError) as e:
            stree.stree_set_wait_hook(**bad)
        assert e.value.status == 1, bad
    for bad in (-1, 1 << 64):                  # would wrap in 64 bits
        with pytest.raises(ValueError):
            stree.stree_set_wait_hook(bad)
    stree.stree_set_wait_hook(2_000_000, 1)
    stree.stree_set_wait_hook()
