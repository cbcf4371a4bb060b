"""Pins of the fp64 definitions in oracle/prompt.py: hand-worked cases, and agreement with
the tree oracles where a chain makes them the same thing."""
import math

import numpy as np
import torch

from hybrid_packed_tree_b200 import workloads as wl
from oracle import oracle_gdn_commit, oracle_gdn_tree, oracle_tree_attention
from oracle.prompt import (oracle_cache_row, oracle_decode_attention, oracle_linear, oracle_pages,
                           oracle_prompt_attention)


def test_linear_by_hand():
    # One head, a 1 x 1 state: S = 2, then 0.5 * 2 + 3 * 2 * 1 = 7, then 0 * 7 + 1 * 4 * 0.5 = 2.
    q = np.array([1.0, 2.0]).reshape(2, 1, 1)
    k = np.array([1.0, 0.5]).reshape(2, 1, 1)
    v = np.array([2.0, 4.0]).reshape(2, 1, 1)
    o, S, oa, Sa = oracle_linear(q, k, v, [[0.5], [0.0]], [[3.0], [1.0]], skip=[10.0], S0=np.full((1, 1, 1), 2.0))
    assert o.ravel().tolist() == [7.0 + 20.0, 4.0 + 40.0]
    assert S.item() == 2.0 and Sa.item() == 2.0 and oa.ravel().tolist() == [27.0, 44.0]


def test_linear_is_the_tree_recurrence_without_erase_on_a_chain():
    T = 9
    parent = wl.chain_tree(T)[None]
    a = wl.gdn_inputs(parent, np.arange(T, dtype=np.int32)[None], np.array([T], np.int32), heads_v=4, heads_k=2, dk=16,
                      dv=8, dtype="f32")
    f = a.f64()
    zero = np.zeros_like(f["beta"])
    o_tree = oracle_gdn_tree(f["q"], f["k"], f["v"], f["alpha"], f["beta"], f["S0"], parent, erase=zero)
    S_tree = oracle_gdn_commit(f["k"], f["v"], f["alpha"], f["beta"], f["S0"], parent, a.path, a.path_len, erase=zero)
    o, S, _, _ = oracle_linear(f["q"][0], f["k"][0], f["v"][0], f["alpha"][0], f["beta"][0], S0=f["S0"][0])
    S_tree = S_tree[0] if isinstance(S_tree, tuple) else S_tree
    np.testing.assert_allclose(o, o_tree[0], rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(S, S_tree[0], rtol=1e-12, atol=1e-12)


def test_prompt_attention_is_tree_attention_on_a_chain():
    rng = np.random.default_rng(3)
    T = 7
    q, k, v = rng.normal(size=(T, 4, 8)), rng.normal(size=(T, 2, 8)), rng.normal(size=(T, 2, 8))
    none = np.zeros((1, 0, 2, 8))
    tree = oracle_tree_attention(q[None], none, none, k[None], v[None], wl.chain_tree(T)[None], 0.3)
    o, oa = oracle_prompt_attention(q, k, v, 0.3)
    np.testing.assert_allclose(o, tree[0], rtol=1e-12, atol=1e-12)
    assert (oa >= np.abs(o) - 1e-12).all()
    last, _ = oracle_decode_attention(q[-1], k, v, 0.3)
    np.testing.assert_allclose(last, o[-1], rtol=1e-12, atol=1e-12)


def test_decode_over_nothing_is_zero():
    o, _ = oracle_decode_attention(np.ones((2, 4)), np.zeros((0, 1, 4)), np.zeros((0, 1, 4)), 1.0)
    assert not o.any()


def test_pages_are_followed_in_table_order():
    pages = np.arange(3 * 1 * 2 * 1, dtype=np.float64).reshape(3, 1, 2, 1)
    assert oracle_pages(pages, [2, 0], 3).ravel().tolist() == [4.0, 5.0, 0.0]


def test_cache_row_by_hand():
    # 448 needs scale 1; a hair above needs 2; 3.5 = 448 / 128.
    assert oracle_cache_row([448.0, 1.0])[0] == 127
    assert oracle_cache_row([450.0, 1.0])[0] == 128
    s, x = oracle_cache_row([3.5, 3.3, -0.01, 0.0])
    assert s == 120 and x[0] == 3.5 and x[3] == 0.0
    assert x[1] == 3.25                       # 422.4 lies between 416 and 448
    assert x[2] == -1.25 / 128                # 1.28 lies between 1.25 and 1.375
    assert oracle_cache_row([0.0, 0.0])[0] == 9
    s, x = oracle_cache_row([math.inf, 2.0, math.nan, -math.inf])
    assert s == 120 and x[0] == 3.5 and x[1] == 2.0 and math.isnan(x[2]) and x[3] == -3.5


def test_cache_row_rounds_as_the_e4m3_type():
    rng = np.random.default_rng(5)
    x = torch.from_numpy(rng.normal(size=512) * np.exp(rng.normal(size=512) * 3)).bfloat16().double().numpy()
    s, got = oracle_cache_row(x)
    y = torch.from_numpy(x * 2.0 ** (127 - s)).float().to(torch.float8_e4m3fn).double().numpy() * 2.0 ** (s - 127)
    np.testing.assert_array_equal(got, y)
