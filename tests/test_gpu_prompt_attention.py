"""Causal attention over packed prompts (stree_prompt_attention) against the fp64
definition: lengths about the tile edges, head groups (powers of two and others), a
neighbour sequence of NaN, rows behind the last sequence, scores that grow along the keys
(the running maximum moves), error words, graphs."""
import numpy as np
import pytest
import torch

from oracle.prompt import oracle_prompt_attention

from prompt_util import attention_tol, bf16, f64, i32, offsets, within

pytestmark = pytest.mark.gpu
SCALE = 0.09


@pytest.fixture(scope="module")
def st():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from hybrid_packed_tree_b200 import stree
    return stree


def _inputs(lens, hq, hkv, seed, extra=0, grow=0.0):
    rng = np.random.default_rng(seed)
    n = int(sum(lens)) + extra
    q, k, v = (rng.normal(size=(n, h, 128)) for h in (hq, hkv, hkv))
    if grow:
        q, k = np.abs(q), k + grow * np.arange(n)[:, None, None] / max(n, 1)
    return dict(q=bf16(q), k=bf16(k), v=bf16(v), cu=i32(offsets(lens)))


def _run(st, a):
    o = torch.full_like(a["q"], 7.0)
    err = torch.full((4,), -1, dtype=torch.int32, device="cuda")
    st.stree_prompt_attention(a["q"], a["k"], a["v"], a["cu"], o, SCALE, err_out=err)
    torch.cuda.synchronize()
    return o, err.tolist()


def _check(a, o, lo, hi, what):
    q, k, v = (f64(a[n][lo:hi]) for n in ("q", "k", "v"))
    ref, oa = oracle_prompt_attention(q, k, v, SCALE)
    rep = q.shape[1] // k.shape[1]
    score = SCALE * np.max(np.einsum("thd,shd->ths", np.abs(q), np.abs(np.repeat(k, rep, 1)))) if hi > lo else 0.0
    within(f64(o[lo:hi]), ref, attention_tol(ref, oa, score), what)


CASES = [
    ([1], 4, 1), ([37], 32, 8), ([32, 33, 1], 4, 1), ([127, 0, 128, 129], 2, 1), ([255, 256, 257], 1, 1),
    ([300, 5, 70], 3, 1), ([130], 5, 1), ([90, 41], 16, 2), ([20], 128, 1), ([64, 2], 100, 1), ([700], 2, 2),
    ([385, 511], 8, 4), ([2] * 40, 4, 2),
]


@pytest.mark.parametrize("lens,hq,hkv", CASES)
def test_prompt_attention_matches_the_definition(st, lens, hq, hkv):
    a = _inputs(lens, hq, hkv, seed=sum(lens) + hq)
    o, err = _run(st, a)
    assert err == [0, 0, 0, 0]
    at = a["cu"].tolist()
    for b, (lo, hi) in enumerate(zip(at, at[1:])):
        _check(a, o, lo, hi, f"sequence {b}")


def test_prompt_attention_moving_maximum(st):
    a = _inputs([520, 130], 4, 2, seed=3, grow=12.0)
    o, err = _run(st, a)
    assert err == [0, 0, 0, 0]
    _check(a, o, 0, 520, "growing scores")
    _check(a, o, 520, 650, "growing scores")


@pytest.mark.parametrize("count,longest,hq,hkv", [(300, 40, 4, 2), (129, 700, 8, 8), (515, 3, 6, 2), (5, 1300, 16, 8)])
def test_prompt_attention_many_tiles(st, count, longest, hq, hkv):
    # More sequences than a warp's group of them, empty ones among them, and more tiles than SMs.
    rng = np.random.default_rng(count)
    lens = rng.integers(0, longest + 1, count)
    lens[0], lens[-1] = longest, 0
    a = _inputs(lens, hq, hkv, seed=count)
    o, err = _run(st, a)
    assert err == [0, 0, 0, 0]
    at = a["cu"].tolist()
    picks = set(rng.choice(count, min(count, 12), replace=False).tolist()) | {0, count - 2, count - 1}
    for b in sorted(picks):
        lo, hi = at[b], at[b + 1]
        if hi - lo > 1000:                     # of two query heads that share no keys
            rep = hq // hkv
            some = dict(q=a["q"][:, ::rep][:, :2], k=a["k"][:, :2], v=a["v"][:, :2])
            _check(some, o[:, ::rep][:, :2], lo, hi, f"sequence {b}")
        else:
            _check(a, o, lo, hi, f"sequence {b}")
    assert torch.isfinite(o.float()).all()
    # The same call twice gives the same bits: which CTA takes a tile does not enter its result.
    o2, _ = _run(st, a)
    assert torch.equal(o, o2)


def test_prompt_attention_keeps_to_its_sequences(st):
    a = _inputs([100, 60, 333], 4, 1, seed=4, extra=40)
    for n in ("q", "k", "v"):
        a[n][100:160] = float("nan")
        a[n][493:] = float("inf")
    o, err = _run(st, a)
    assert err == [0, 0, 0, 0]
    _check(a, o, 0, 100, "before NaN")
    _check(a, o, 160, 493, "behind NaN")
    assert torch.all(o[493:] == 7.0)


def test_prompt_attention_bad_offsets(st):
    a = _inputs([50, 20, 30], 4, 1, seed=5)
    a["cu"] = i32([0, 50, 45, 101])
    o, err = _run(st, a)
    assert err[0] == 9 and err[1] in (1, 2)
    _check(a, o, 0, 50, "beside bad offsets")
    assert torch.all(o[50:] == 7.0)


def test_prompt_attention_no_rows_and_no_error_word(st):
    a = _inputs([0, 0], 4, 1, seed=6)
    o, err = _run(st, a)
    assert err == [0, 0, 0, 0] and o.numel() == 0
    a = _inputs([77], 4, 1, seed=7)
    o = torch.empty_like(a["q"])
    st.stree_prompt_attention(a["q"], a["k"], a["v"], a["cu"], o, SCALE)
    torch.cuda.synchronize()
    _check(a, o, 0, 77, "no error word")


def test_prompt_attention_in_a_graph_and_on_another_stream(st):
    a = _inputs([200, 61], 8, 2, seed=8)
    o = torch.empty_like(a["q"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        st.stree_prompt_attention(a["q"], a["k"], a["v"], a["cu"], o, SCALE)
    torch.cuda.current_stream().wait_stream(s)
    want = o.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        st.stree_prompt_attention(a["q"], a["k"], a["v"], a["cu"], o, SCALE)
    b = _inputs([200, 61], 8, 2, seed=9)
    for n in ("q", "k", "v"):
        a[n].copy_(b[n])
    g.replay()
    torch.cuda.synchronize()
    assert not torch.equal(o, want)
    _check(a, o, 0, 200, "replayed")
    _check(a, o, 200, 261, "replayed")


def test_prompt_attention_output_at_a_16_byte_boundary(st):
    a = _inputs([140, 33], 8, 2, seed=10)
    n = a["q"].numel()
    room = torch.full((n + 16,), 7.0, dtype=torch.bfloat16, device="cuda")
    o = room[8:8 + n].view(a["q"].shape)
    assert o.data_ptr() % 32 == 16
    st.stree_prompt_attention(a["q"], a["k"], a["v"], a["cu"], o, SCALE)
    torch.cuda.synchronize()
    _check(a, o, 0, 140, "first sequence")
    _check(a, o, 140, 173, "second sequence")
    assert torch.all(room[:8] == 7.0) and torch.all(room[-8:] == 7.0)
