"""The calls together, as a server of a hybrid model uses them: prompts through a
linear-attention layer and an attention layer, their cache written into pages, single
tokens, then a draft tree verified from the state and the cache that these left, its
accepted path committed, and one more token.  Everything is checked against the fp64
definitions over the whole sequences."""
import numpy as np
import pytest
import torch

from oracle import oracle_gdn_tree, oracle_tree_attention
from oracle.prompt import oracle_decode_attention, oracle_linear, oracle_prompt_attention

from hybrid_packed_tree_b200 import workloads as wl
from prompt_util import U, attention_tol, bf16, f32, f64, i32, offsets, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def st():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from hybrid_packed_tree_b200 import stree
    return stree


def test_attention_layer_from_prompt_to_tree(st):
    rng = np.random.default_rng(1)
    lens, hq, hkv, page, scale = [70, 130], 8, 2, 16, 0.09
    n, b = sum(lens), len(lens)
    q, k, v = bf16(rng.normal(size=(n, hq, 128))), bf16(rng.normal(size=(n, hkv, 128))), bf16(rng.normal(size=(n, hkv, 128)))
    err = torch.zeros(4, dtype=torch.int32, device="cuda")
    o = torch.empty_like(q)
    cu = i32(offsets(lens))
    st.stree_prompt_attention(q, k, v, cu, o, scale, err_out=err)
    for i, (lo, hi) in enumerate(zip([0, 70], [70, 200])):
        ref, oa = oracle_prompt_attention(f64(q[lo:hi]), f64(k[lo:hi]), f64(v[lo:hi]), scale)
        within(f64(o[lo:hi]), ref, attention_tol(ref, oa, 40.0), f"prompt {i}")
    # The cache: room for 12 pages each; the prompt, one decoded token, a tree's path, one more token.
    table = i32(rng.permutation(24).reshape(2, 12))
    kp = torch.full((24, hkv, page, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    vp = torch.full_like(kp, float("nan"))
    ws = torch.empty(st.stree_paged_attention_workspace_size(hq, hkv), dtype=torch.uint8, device="cuda")
    st.stree_cache_write(k, v, cu, i32([0, 0]), table, kp, vp, err_out=err)
    hist_k = [f64(k[:70]), f64(k[70:])]
    hist_v = [f64(v[:70]), f64(v[70:])]

    def token(seed):
        r = np.random.default_rng(seed)
        q1, k1, v1 = bf16(r.normal(size=(b, hq, 128))), bf16(r.normal(size=(b, hkv, 128))), bf16(r.normal(size=(b, hkv, 128)))
        held = [len(h) for h in hist_k]
        st.stree_cache_write(k1, v1, i32([0, 1, 2]), i32(held), table, kp, vp, err_out=err)
        o1 = torch.empty_like(q1)
        st.stree_paged_attention(q1, kp, vp, table, i32([h + 1 for h in held]), o1, scale, err_out=err, workspace=ws)
        for s in range(b):
            hist_k[s] = np.concatenate([hist_k[s], f64(k1[s:s + 1])])
            hist_v[s] = np.concatenate([hist_v[s], f64(v1[s:s + 1])])
            ref, oa = oracle_decode_attention(f64(q1[s]), hist_k[s], hist_v[s], scale)
            within(f64(o1[s]), ref, attention_tol(ref, oa, 40.0), f"token of sequence {s}")

    token(2)
    # A draft tree over the contiguous reading of the cache, and the commit of its path.
    parent = np.array([wl.M2_PARENT_15] * b, np.int32)
    a = wl.attention_inputs(parent, 0, [0] * b, heads_q=hq, heads_kv=hkv, seed=3)
    qt, kt, vt = (torch.from_numpy(a[x].view(np.int16)).view(torch.bfloat16).cuda() for x in ("q", "k_tree", "v_tree"))
    held = [len(h) for h in hist_k]
    kc = torch.full((b, 160, hkv, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc = torch.full_like(kc, float("nan"))
    st.stree_cache_read(kp, vp, table, i32(held), kc, vc, err_out=err)
    ot = torch.empty_like(qt)
    tree_err = torch.zeros(4, dtype=torch.int32, device="cuda")
    st.stree_tree_attention(qt, kc, vc, kt, vt, i32(held), i32(parent), ot, scale, tree_err)
    path, plen = i32([[0, 1, 4, 10], [0, 3, -1, -1]]), i32([4, 2])
    st.stree_cache_commit(kt, vt, path, plen, i32(held), table, kp, vp, err_out=err)
    torch.cuda.synchronize()
    for s in range(b):
        ref = oracle_tree_attention(f64(qt[s:s + 1]), hist_k[s][None], hist_v[s][None], f64(kt[s:s + 1]), f64(vt[s:s + 1]),
                                    parent[s:s + 1], scale)
        within(f64(ot[s:s + 1]), ref, 2e-2 * np.abs(ref).max(), f"tree of sequence {s}")
        for i in range(int(plen[s])):
            node = int(path[s, i])
            hist_k[s] = np.concatenate([hist_k[s], f64(kt[s, node:node + 1])])
            hist_v[s] = np.concatenate([hist_v[s], f64(vt[s, node:node + 1])])
    token(5)
    torch.cuda.synchronize()
    assert err.tolist() == [0, 0, 0, 0] and tree_err.tolist() == [0, 0, 0, 0]


def test_linear_layer_from_prompt_to_tree(st):
    rng = np.random.default_rng(7)
    lens, hv, hk = [140, 33], 4, 2
    n, b = sum(lens) + 2, 2                    # two prompts, then a token each
    a = wl.gdn_inputs(wl.chain_tree(n)[None], np.zeros((1, 1), np.int32), np.ones(1, np.int32), heads_v=hv, heads_k=hk, seed=8)
    q, k, v = (torch.from_numpy(getattr(a, x)[0].view(np.int16)).view(torch.bfloat16).cuda() for x in ("q", "k", "v"))
    alpha, beta = f32(a.alpha[0]), f32(a.beta[0])
    S = torch.empty(b, hv, 128, 128, device="cuda")
    o = torch.empty_like(v)
    err = torch.zeros(4, dtype=torch.int32, device="cuda")
    st.stree_linear_prompt(q, k, v, alpha, beta, i32(offsets(lens)), o, S_new=S, err_out=err)
    tail = slice(173, 175)
    o1 = torch.empty_like(v[tail])
    st.stree_linear_step(q[tail], k[tail], v[tail], alpha[tail], beta[tail], S, o1, S)
    parent = np.array([wl.M2_PARENT_15] * b, np.int32)
    t = wl.gdn_inputs(parent, np.zeros((b, 1), np.int32), np.ones(b, np.int32), heads_v=hv, heads_k=hk, seed=9)
    qt, kt, vt = (torch.from_numpy(getattr(t, x).view(np.int16)).view(torch.bfloat16).cuda() for x in ("q", "k", "v"))
    ot = torch.empty_like(vt)
    zero = torch.zeros(b, 15, hv, device="cuda")
    tree_err = torch.zeros(4, dtype=torch.int32, device="cuda")
    st.stree_gdn_tree_scan_commit(qt, kt, vt, f32(t.alpha), f32(t.beta), S, i32(parent), ot, err_out=tree_err, erase=zero)
    torch.cuda.synchronize()
    assert err.tolist() == [0, 0, 0, 0] and tree_err.tolist() == [0, 0, 0, 0]
    f = t.f64()
    for s, (lo, hi) in enumerate(((0, 140), (140, 173))):
        rows = list(range(lo, hi)) + [173 + s]
        ro, rS, oa, Sa = oracle_linear(f64(q[rows]), f64(k[rows]), f64(v[rows]), f64(alpha[rows]), f64(beta[rows]))
        got = np.concatenate([f64(o[lo:hi]), f64(o1[s:s + 1])])
        within(got, ro, U * np.abs(ro) + (U + 2.0 ** -12) * oa, f"outputs of sequence {s}")
        within(f64(S[s]), rS, 2.0 ** -13 * Sa, f"state of sequence {s}")
        rt = oracle_gdn_tree(f["q"][s:s + 1], f["k"][s:s + 1], f["v"][s:s + 1], f["alpha"][s:s + 1], f["beta"][s:s + 1], rS[None],
                             parent[s:s + 1], erase=np.zeros((1, 15, hv)))
        within(f64(ot[s:s + 1]), rt, 2e-2 * np.abs(rt).max(), f"tree of sequence {s}")
