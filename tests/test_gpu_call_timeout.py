"""Failure detection of the warp-role kernels without a context, exercised without a GPU fault.

Their waits are bounded.  The test hook withholds one hand-off between two roles, on which no
copy depends, so that a wait runs out: the call must return, report STREE_ERR_TIMEOUT in the
error word whichever role gave up, leave what it did not compute untouched, and the next call
must be exact again.
"""
import numpy as np
import pytest
import torch

from oracle.prompt import oracle_decode_attention, oracle_linear, oracle_pages, oracle_prompt_attention

from prompt_util import E, U, attention_tol, bf16, f32, f64, i32, offsets, random_tables, within

pytestmark = pytest.mark.gpu

STREE_ERR_TIMEOUT = 7
SCALE = 0.09


@pytest.fixture(scope="module")
def st():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from hybrid_packed_tree_b200 import stree
    return stree


@pytest.fixture
def fault(st):
    """Runs a call with the hook set: its error word."""
    def run(call):
        err = torch.full((4,), -1, dtype=torch.int32, device="cuda")
        st.stree_set_wait_hook(2_000_000, 1)   # 2 ms
        try:
            call(err)
        finally:
            st.stree_set_wait_hook()
        torch.cuda.synchronize()
        return err.tolist()
    yield run
    st.stree_set_wait_hook()


@pytest.mark.parametrize("lens", [[1], [97], [300, 0, 5], [700, 650]])
def test_prompt_attention_reports_a_wait_that_ran_out(st, fault, lens):
    rng = np.random.default_rng(sum(lens))
    n = sum(lens)
    q, k, v = (bf16(rng.normal(size=(n, h, 128))) for h in (4, 2, 2))
    cu = i32(offsets(lens))
    o = torch.full_like(q, 7.0)
    err = fault(lambda e: st.stree_prompt_attention(q, k, v, cu, o, SCALE, err_out=e))
    assert err[0] == STREE_ERR_TIMEOUT, err
    assert torch.all(o == 7.0)                 # every CTA gave up at its first tile
    err = torch.full((4,), -1, dtype=torch.int32, device="cuda")
    st.stree_prompt_attention(q, k, v, cu, o, SCALE, err_out=err)
    torch.cuda.synchronize()
    assert err.tolist() == [0, 0, 0, 0]
    at = offsets(lens)
    for lo, hi in zip(at, at[1:]):
        ref, oa = oracle_prompt_attention(f64(q[lo:hi]), f64(k[lo:hi]), f64(v[lo:hi]), SCALE)
        within(f64(o[lo:hi]), ref, attention_tol(ref, oa, 40.0), "after the timeout")


@pytest.mark.parametrize("dv", [128, 64])
@pytest.mark.parametrize("lens", [[1], [128, 0, 129], [2300, 1900, 5]])
def test_linear_prompt_reports_a_wait_that_ran_out(st, fault, lens, dv):
    """One chunk (the gate warp is done long before another role gives up), several, and the split."""
    rng = np.random.default_rng(sum(lens))
    n, b, hv, hk = sum(lens), len(lens), 2, 1
    q, k = (bf16(rng.normal(size=(n, hk, 128)) / np.sqrt(128)) for _ in range(2))
    v, alpha, beta = bf16(rng.normal(size=(n, hv, dv))), f32(rng.uniform(0.9, 1.0, size=(n, hv))), f32(rng.uniform(size=(n, hv)))
    S0, cu = f32(rng.normal(0, 0.3, size=(b, hv, dv, 128))), i32(offsets(lens))
    ws = torch.full((max(16, st.stree_linear_prompt_workspace_size(b, n, hv, hk, 128, dv)),), 0xFF, dtype=torch.uint8, device="cuda")
    o, S = torch.full_like(v, 7.0), torch.full_like(S0, 7.0)

    def call(err):
        st.stree_linear_prompt(q, k, v, alpha, beta, cu, o, S0=S0, S_new=S, err_out=err, workspace=ws)

    err = fault(call)
    assert err[0] == STREE_ERR_TIMEOUT, err
    assert torch.all(o == 7.0)                 # every CTA gave up at its first chunk
    err = torch.full((4,), -1, dtype=torch.int32, device="cuda")
    call(err)
    torch.cuda.synchronize()
    assert err.tolist() == [0, 0, 0, 0]
    at = offsets(lens)
    for i, (lo, hi) in enumerate(zip(at, at[1:])):
        ro, rS, oa, Sa = oracle_linear(*(f64(t[lo:hi]) for t in (q, k, v, alpha, beta)), S0=f64(S0[i]))
        ops = 2 * (hi - lo) + 128 + 300        # as for the prompts without a timeout
        within(f64(o[lo:hi]), ro, U * np.abs(ro) + (U + ops * E) * oa + 1e-30, "o after the timeout")
        within(f64(S[i]), rS, ops * E * Sa + 1e-30, "S after the timeout")


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,hq", [([1], 4), ([40, 0, 5], 8), ([9000, 700], 24)])
def test_paged_attention_reports_a_wait_that_ran_out(st, fault, lens, hq, cache):
    """Shares that fit in the ring of stages (the producer is done when the others give up) and longer ones."""
    rng = np.random.default_rng(sum(lens) + hq)
    hkv, page = 2, 16
    table, n_pages = random_tables(rng, lens, page)
    pages, scales, values = [], [], []
    for _ in range(2):
        x = bf16(rng.normal(size=(n_pages, hkv, page, 128)))
        pages.append(x if cache == "bf16" else x.float().to(torch.float8_e4m3fn))
        scales.append(None if cache == "bf16" else torch.full((n_pages, hkv, page), 127, dtype=torch.uint8, device="cuda"))
        values.append(f64(pages[-1].float()))
    q = bf16(rng.normal(size=(len(lens), hq, 128)))
    ws = torch.full((st.stree_paged_attention_workspace_size(hq, hkv),), 0xFF, dtype=torch.uint8, device="cuda")
    o, tab, n = torch.full_like(q, 7.0), i32(table), i32(lens)

    def call(err):
        st.stree_paged_attention(q, *pages, tab, n, o, SCALE, k_scales=scales[0], v_scales=scales[1], err_out=err, workspace=ws)

    err = fault(call)
    assert err[0] == STREE_ERR_TIMEOUT, err
    for b, length in enumerate(lens):          # every share gave up at its first block
        assert torch.all(o[b] == (7.0 if length else 0.0))
    err = torch.full((4,), -1, dtype=torch.int32, device="cuda")
    call(err)
    torch.cuda.synchronize()
    assert err.tolist() == [0, 0, 0, 0]
    for b, length in enumerate(lens):
        k, v = (oracle_pages(x, table[b], length) for x in values)
        ref, oa = oracle_decode_attention(f64(q[b]), k, v, SCALE)
        within(f64(o[b]), ref, attention_tol(ref, oa, 40.0), "after the timeout")


@pytest.mark.parametrize("more", [0, 40])
def test_linear_prompt_keeps_what_its_first_blocks_report(st, fault, more):
    """As many CTAs as SMs give up, and more wait behind them: the block that clears the error word does not."""
    n = torch.cuda.get_device_properties(0).multi_processor_count + more
    rng = np.random.default_rng(n)
    q, k, v = (bf16(rng.normal(size=(n, 1, 128))) for _ in range(3))
    alpha, cu = f32(np.ones((n, 1))), i32(np.minimum(np.arange(n + 1), n - more))    # the last are empty
    o = torch.full_like(v, 7.0)
    err = fault(lambda e: st.stree_linear_prompt(q, k, v, alpha, None, cu, o, err_out=e))
    assert err[0] == STREE_ERR_TIMEOUT, err
    assert torch.all(o == 7.0)
    err = torch.full((4,), -1, dtype=torch.int32, device="cuda")
    st.stree_linear_prompt(q, k, v, alpha, None, cu, o, err_out=err)
    torch.cuda.synchronize()
    assert err.tolist() == [0, 0, 0, 0]
    ref = (f64(q) * f64(k)).sum(-1, keepdims=True) * f64(v)                          # one token each, from no state
    oa = (np.abs(f64(q)) * np.abs(f64(k))).sum(-1, keepdims=True) * np.abs(f64(v))
    rows = n - more
    within(f64(o[:rows]), ref[:rows], (U * np.abs(ref) + (U + 430 * E) * oa + 1e-30)[:rows], "after the timeout")
    assert torch.all(o[rows:] == 7.0)


def test_paged_attention_keeps_what_its_first_blocks_report(st, fault):
    """More sequences than CTAs fit on the GPU: every CTA gives up, and the block that clears the error word is not the last."""
    n = 3 * torch.cuda.get_device_properties(0).multi_processor_count
    rng = np.random.default_rng(n)
    pages = [bf16(rng.normal(size=(n, 1, 8, 128))) for _ in range(2)]
    q, table, lens = bf16(rng.normal(size=(n, 2, 128))), i32(np.arange(n)[:, None]), i32(np.full(n, 8))
    ws = torch.full((st.stree_paged_attention_workspace_size(2, 1),), 0xFF, dtype=torch.uint8, device="cuda")
    o = torch.full_like(q, 7.0)
    err = fault(lambda e: st.stree_paged_attention(q, *pages, table, lens, o, SCALE, err_out=e, workspace=ws))
    assert err[0] == STREE_ERR_TIMEOUT, err
    assert torch.all(o == 7.0)
    err = torch.full((4,), -1, dtype=torch.int32, device="cuda")
    st.stree_paged_attention(q, *pages, table, lens, o, SCALE, err_out=err, workspace=ws)
    torch.cuda.synchronize()
    assert err.tolist() == [0, 0, 0, 0]
    for b in range(n):
        ref, oa = oracle_decode_attention(f64(q[b]), f64(pages[0][b]).transpose(1, 0, 2), f64(pages[1][b]).transpose(1, 0, 2), SCALE)
        within(f64(o[b]), ref, attention_tol(ref, oa, 40.0), "after the timeout")
