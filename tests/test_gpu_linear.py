"""Linear attention with a decay for each head (stree_linear_prompt, stree_linear_step)
against the token-by-token definition in fp64: both types, packed sequences of lengths from
none up over several chunks, head groups, state shapes of every path, decays of zero,
rows behind the last sequence, other sequences' NaN, error words, and the split over a
workspace."""
import numpy as np
import pytest
import torch

from oracle.prompt import oracle_linear

from prompt_util import E, U, bf16, f32, f64, i32, offsets, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def st():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from hybrid_packed_tree_b200 import stree
    return stree


def _inputs(lens, hv, hk, dk, dv, dtype, seed, *, skip=True, start=True, beta=True, extra=0, decay=None):
    rng = np.random.default_rng(seed)
    n = int(sum(lens)) + extra
    up = bf16 if dtype == "bf16" else f32
    a = dict(q=up(rng.normal(size=(n, hk, dk)) / np.sqrt(dk)), k=up(rng.normal(size=(n, hk, dk)) / np.sqrt(dk)),
             v=up(rng.normal(size=(n, hv, dv))))
    rate = np.exp(rng.uniform(np.log(1e-3), np.log(4.0), size=hv)) if decay is None else decay
    a["alpha"] = f32(np.exp(-rate * np.logaddexp(0.0, rng.normal(-1.0, 0.5, size=(n, hv)))))
    a["beta"] = f32(1 / (1 + np.exp(-rng.normal(size=(n, hv))))) if beta else None
    a["skip"] = f32(rng.normal(size=hv)) if skip else None
    a["S0"] = f32(rng.normal(0, 0.3, size=(len(lens), hv, dv, dk))) if start else None
    a["cu"] = i32(offsets(lens))
    return a


def _run(st, a, split=True, in_place=False):
    b, (hv, dv), dk = a["cu"].shape[0] - 1, a["v"].shape[1:], a["k"].shape[2]
    o = torch.full_like(a["v"], 7.0)
    S = a["S0"].clone() if in_place else torch.full((b, hv, dv, dk), 7.0, device="cuda")
    err = torch.full((4,), -1, dtype=torch.int32, device="cuda")
    size = st.stree_linear_prompt_workspace_size(b, a["v"].shape[0], hv, a["k"].shape[1], dk, dv, a["v"].dtype)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda") if split and size else None
    st.stree_linear_prompt(a["q"], a["k"], a["v"], a["alpha"], a["beta"], a["cu"], o, S0=S if in_place else a["S0"], S_new=S,
                           skip=a["skip"], err_out=err, workspace=ws)
    torch.cuda.synchronize()
    return o, S, err.tolist()


def _check(a, o, S, what):
    """fp32: 2 operations a token into a state, dk into an output.  bf16 adds the output's rounding
    and, per term, that of a pair weight or of a state that a query reads."""
    at = a["cu"].tolist()
    g = lambda n, lo, hi: None if a[n] is None else f64(a[n][lo:hi])  # noqa: E731
    for b, (lo, hi) in enumerate(zip(at, at[1:])):
        ro, rS, oa, Sa = oracle_linear(g("q", lo, hi), g("k", lo, hi), g("v", lo, hi), g("alpha", lo, hi), g("beta", lo, hi),
                                       skip=None if a["skip"] is None else f64(a["skip"]),
                                       S0=None if a["S0"] is None else f64(a["S0"][b]))
        ops = 2 * (hi - lo) + a["k"].shape[2] + 300
        u = U if a["v"].dtype == torch.bfloat16 else 0.0
        within(f64(o[lo:hi]), ro, u * np.abs(ro) + (u + ops * E) * oa + 1e-30, f"{what} o of sequence {b}")
        within(f64(S[b]), rS, ops * E * Sa + 1e-30, f"{what} S of sequence {b}")


CASES = [
    # (lengths, value heads, key heads, dk, dv, dtype)
    ([1], 2, 1, 128, 128, "bf16"),
    ([127], 4, 2, 128, 128, "bf16"),
    ([128, 0, 129], 2, 2, 128, 128, "bf16"),
    ([300, 1, 64, 513], 4, 1, 128, 128, "bf16"),
    ([1, 37, 256, 2], 6, 1, 128, 64, "bf16"),
    ([640], 4, 2, 128, 64, "bf16"),
    ([130, 5], 5, 5, 128, 64, "bf16"),         # an odd group of 64-wide heads
    ([200], 3, 1, 128, 96, "bf16"),
    ([70, 3], 2, 1, 64, 32, "bf16"),
    ([50], 2, 2, 256, 256, "bf16"),
    ([1, 0, 40], 2, 1, 128, 128, "f32"),
    ([129, 33], 4, 2, 64, 32, "f32"),
    ([17], 3, 3, 8, 8, "f32"),
    ([21, 2], 2, 1, 136, 40, "f32"),
]


@pytest.mark.parametrize("lens,hv,hk,dk,dv,dtype", CASES)
def test_prompt_matches_the_definition(st, lens, hv, hk, dk, dv, dtype):
    a = _inputs(lens, hv, hk, dk, dv, dtype, seed=len(lens) * 100 + hv)
    o, S, err = _run(st, a)
    assert err == [0, 0, 0, 0]
    _check(a, o, S, "prompt")


@pytest.mark.parametrize("dv", [128, 64])
@pytest.mark.parametrize("skip,start,beta", [(False, True, True), (True, False, True), (False, False, False)])
def test_prompt_without_the_optional_inputs(st, dv, skip, start, beta):
    a = _inputs([140, 9], 2, 1, 128, dv, "bf16", seed=5, skip=skip, start=start, beta=beta)
    o, S, err = _run(st, a)
    assert err == [0, 0, 0, 0]
    _check(a, o, S, "prompt")


@pytest.mark.parametrize("dv", [128, 64])
def test_prompt_split_over_the_long_axis(st, dv):
    lens = [2300, 1900, 5]
    a = _inputs(lens, 2, 1, 128, dv, "bf16", seed=8, decay=np.array([1e-3, 0.02]))
    assert st.stree_linear_prompt_workspace_size(len(lens), sum(lens), 2, 1, 128, dv) > 0
    whole = _run(st, a, split=False)
    split = _run(st, a, split=True)
    assert whole[2] == split[2] == [0, 0, 0, 0]
    _check(a, *whole[:2], "unsplit")
    _check(a, *split[:2], "split")
    inp = _run(st, a, split=True, in_place=True)
    assert torch.equal(inp[0], split[0]) and torch.equal(inp[1], split[1])


@pytest.mark.parametrize("dtype,dv", [("bf16", 128), ("bf16", 64), ("f32", 64)])
def test_prompt_decay_of_zero_forgets(st, dtype, dv):
    a = _inputs([260], 2, 1, 128, dv, dtype, seed=9)
    a["alpha"][[0, 5, 6, 127, 128, 200]] = 0.0
    a["alpha"][:, 1] *= 1e-30                  # every token forgets
    o, S, err = _run(st, a)
    assert err == [0, 0, 0, 0]
    _check(a, o, S, "zero decay")
    b = {k: v for k, v in a.items()}
    b["S0"] = a["S0"] * 1000                   # what was before a zero does not matter
    o2, S2, _ = _run(st, b)
    assert torch.equal(o, o2) and torch.equal(S, S2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_keeps_to_its_sequences(st, dtype):
    """A sequence next to one of NaN, and rows behind the last sequence."""
    a = _inputs([100, 30, 50], 2, 1, 128, 128, dtype, seed=11, extra=20)
    for n in ("q", "k", "v", "alpha"):
        a[n][100:130] = float("nan")
        a[n][180:] = float("nan")
    o, S, err = _run(st, a)
    assert err == [0, 0, 0, 0]
    assert torch.all(o[180:] == 7.0)
    keep = {n: (t if n in ("skip",) else t) for n, t in a.items()}
    for b, (lo, hi) in ((0, (0, 100)), (2, (130, 180))):
        one = {n: (t[lo:hi] if n in ("q", "k", "v", "alpha", "beta") else t) for n, t in keep.items()}
        one["S0"], one["cu"] = a["S0"][b:b + 1], i32([0, hi - lo])
        _check(one, o[lo:hi], S[b:b + 1], "beside NaN")


def test_prompt_in_place_state_and_empty_batch_of_rows(st):
    a = _inputs([150, 0], 2, 1, 128, 128, "bf16", seed=12)
    o, S, _ = _run(st, a)
    o2, S2, _ = _run(st, a, in_place=True)
    assert torch.equal(o, o2) and torch.equal(S, S2)
    assert torch.equal(S[1], a["S0"][1])       # an empty sequence keeps its state
    none = _inputs([0, 0], 2, 1, 128, 128, "bf16", seed=13)
    _, S, err = _run(st, none)
    assert err == [0, 0, 0, 0] and torch.equal(S, none["S0"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_bad_offsets_are_reported_and_skipped(st, dtype):
    a = _inputs([40, 20, 30], 2, 1, 128, 128, dtype, seed=14)
    a["cu"] = i32([0, 40, 30, 90])             # the second sequence's offsets go back
    o, S, err = _run(st, a)
    assert err[:2] == [9, 1]
    assert torch.equal(S[1], a["S0"][1])
    a["cu"] = i32([0, 40, 60, 91])             # past the packed rows
    o, S, err = _run(st, a)
    assert err[:2] == [9, 2]
    one = {n: (t[:40] if n in ("q", "k", "v", "alpha", "beta") else t) for n, t in a.items()}
    one["S0"], one["cu"] = a["S0"][:1], i32([0, 40])
    _check(one, o[:40], S[:1], "beside bad offsets")


STEPS = [(1, 80, 1, 128, 64, "bf16"), (3, 4, 2, 128, 128, "bf16"), (2, 3, 3, 64, 40, "f32"), (5, 2, 1, 256, 8, "f32"),
         (1, 1, 1, 8, 8, "bf16"), (2, 2, 1, 136, 256, "bf16")]


@pytest.mark.parametrize("batch,hv,hk,dk,dv,dtype", STEPS)
@pytest.mark.parametrize("in_place", [False, True])
def test_step_matches_the_definition(st, batch, hv, hk, dk, dv, dtype, in_place):
    a = _inputs([1] * batch, hv, hk, dk, dv, dtype, seed=21 + batch, skip=batch != 3, beta=batch != 5)
    o = torch.full_like(a["v"], 7.0)
    S = a["S0"].clone() if in_place else torch.full_like(a["S0"], 7.0)
    st.stree_linear_step(a["q"], a["k"], a["v"], a["alpha"], a["beta"], S if in_place else a["S0"], o, S, skip=a["skip"])
    torch.cuda.synchronize()
    _check(a, o, S, "step")


def test_steps_continue_a_prompt(st):
    """A prompt, then single tokens, is the whole sequence."""
    a = _inputs([135], 4, 2, 128, 128, "bf16", seed=31)
    head = {n: (t[:130] if n in ("q", "k", "v", "alpha", "beta") else t) for n, t in a.items()}
    head["cu"] = i32([0, 130])
    o, S, _ = _run(st, head)
    outs = [o]
    for t in range(130, 135):
        row = {n: a[n][t:t + 1] for n in ("q", "k", "v", "alpha", "beta")}
        step = torch.empty_like(row["v"])
        st.stree_linear_step(row["q"], row["k"], row["v"], row["alpha"], row["beta"], S, step, S, skip=a["skip"])
        outs.append(step)
    _check(a, torch.cat(outs), S, "prompt and steps")


@pytest.mark.parametrize("dv,lens", [(128, [2300, 1900]), (64, [150, 3])])
def test_prompt_in_a_graph_and_on_another_stream(st, dv, lens):
    """Captured with and without the split, replayed on other inputs; the same bits as an eager call."""
    a = _inputs(lens, 2, 1, 128, dv, "bf16", seed=41)
    o, S = torch.empty_like(a["v"]), torch.empty_like(a["S0"])
    ws = torch.empty(max(16, st.stree_linear_prompt_workspace_size(len(lens), sum(lens), 2, 1, 128, dv)), dtype=torch.uint8,
                     device="cuda")
    err = torch.zeros(4, dtype=torch.int32, device="cuda")

    def call():
        st.stree_linear_prompt(a["q"], a["k"], a["v"], a["alpha"], a["beta"], a["cu"], o, S0=a["S0"], S_new=S, skip=a["skip"],
                               err_out=err, workspace=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    b = _inputs(lens, 2, 1, 128, dv, "bf16", seed=42)
    for n in ("q", "k", "v", "alpha", "beta", "S0", "skip"):
        a[n].copy_(b[n])
    g.replay()
    torch.cuda.synchronize()
    want = _run(st, b)
    assert torch.equal(o, want[0]) and torch.equal(S, want[1]) and err.tolist() == [0, 0, 0, 0]


@pytest.mark.parametrize("dv", [128, 64])
def test_prompt_nan_gates_are_not_hidden(st, dv):
    a = _inputs([200], 2, 1, 128, dv, "bf16", seed=43)
    a["alpha"][150, 0] = float("nan")
    o, S, _ = _run(st, a)
    assert torch.isnan(S[0, 0]).all() and torch.isfinite(S[0, 1]).all() and torch.isfinite(o[:128]).all()
    assert torch.isnan(o[150:, 0]).all() and torch.isfinite(o[:, 1]).all()


def test_prompt_many_short_sequences(st):
    """More sequences than a block has threads, most of them of one token."""
    lens = [1] * 700 + [0, 5, 130]
    a = _inputs(lens, 2, 1, 128, 128, "bf16", seed=44, skip=False)
    o, S, err = _run(st, a)
    assert err == [0, 0, 0, 0]
    at = a["cu"].tolist()
    pick = [0, 1, 399, 699, 700, 701, 702]
    for b in pick:
        lo, hi = at[b], at[b + 1]
        one = {n: (t[lo:hi] if n in ("q", "k", "v", "alpha", "beta") else t) for n, t in a.items()}
        one["S0"], one["cu"] = a["S0"][b:b + 1], i32([0, hi - lo])
        _check(one, o[lo:hi], S[b:b + 1], f"of many, {b}")
