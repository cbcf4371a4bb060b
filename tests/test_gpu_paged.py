"""The paged cache and the attention of one new token over it (stree_paged_attention,
stree_cache_write, stree_cache_commit, stree_cache_read) against the fp64 definitions:
page sizes that end inside a block, head groups beyond a tile, lengths from none up,
stale NaN past a sequence's end, pages out of range, and both page types."""
import numpy as np
import pytest
import torch

from oracle.prompt import oracle_cache_row, oracle_decode_attention, oracle_pages

from prompt_util import attention_tol, bf16, f64, i32, offsets, random_tables, within

pytestmark = pytest.mark.gpu
SCALE = 0.09
BAD = 1 << 30


@pytest.fixture(scope="module")
def st():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from hybrid_packed_tree_b200 import stree
    return stree


def _values(a):
    """What the pages stand for, in fp64: [pages, H, page, 128] each."""
    out = []
    for n in ("k", "v"):
        x = f64(a[n + "_pages"].float())
        if a[n + "_scales"] is not None:
            x = x * 2.0 ** (f64(a[n + "_scales"]) - 127)[..., None]
        out.append(x)
    return out


def _cache(rng, lens, hkv, page, cache, stale=True):
    table, n = random_tables(rng, lens, page)
    a = dict(table=i32(table), lens=i32(lens), k_scales=None, v_scales=None)
    used = np.zeros((n, page), bool)
    for b, ln in enumerate(lens):
        for j in range(ln):
            used[table[b, j // page], j % page] = True
    for name in ("k", "v"):
        x = rng.normal(size=(n, hkv, page, 128)) * np.exp(rng.normal(size=128) * 0.5)
        if stale:
            x[~used[:, None].repeat(hkv, 1)] = np.nan
        if cache == "bf16":
            a[name + "_pages"] = bf16(x)
        else:
            a[name + "_pages"] = torch.from_numpy(x.astype(np.float32) * 16).to(torch.float8_e4m3fn).cuda()
            a[name + "_scales"] = torch.from_numpy(rng.integers(119, 126, size=(n, hkv, page)).astype(np.uint8)).cuda()
    return a


def _attend(st, a, q, err=True, workspace=None):
    o = torch.full_like(q, 7.0)
    e = torch.full((4,), -1, dtype=torch.int32, device="cuda") if err else None
    hkv = a["k_pages"].shape[1]
    if workspace is None:
        size = st.stree_paged_attention_workspace_size(q.shape[1], hkv)
        workspace = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    st.stree_paged_attention(q, a["k_pages"], a["v_pages"], a["table"], a["lens"], o, SCALE, k_scales=a["k_scales"],
                             v_scales=a["v_scales"], err_out=e, workspace=workspace)
    torch.cuda.synchronize()
    return o, e.tolist() if err else None


def _check(a, q, o, keep=None):
    k, v = _values(a)
    table = a["table"].cpu().numpy()
    for b, n in enumerate(a["lens"].tolist()):
        if keep is not None and b not in keep:
            continue
        n = max(0, min(n, table.shape[1] * k.shape[2]))
        kb, vb = oracle_pages(k, table[b], n), oracle_pages(v, table[b], n)
        ref, oa = oracle_decode_attention(f64(q[b]), kb, vb, SCALE)
        rep = q.shape[1] // k.shape[1]
        score = SCALE * np.max(np.einsum("hd,nhd->nh", np.abs(f64(q[b])), np.abs(np.repeat(kb, rep, 1)))) if n else 0.0
        within(f64(o[b]), ref, attention_tol(ref, oa, score), f"sequence {b} of {n}")


CASES = [
    # (lengths, query heads, key/value heads, page size)
    ([1], 4, 1, 8), ([64, 0, 65, 63], 32, 8, 16), ([7, 300, 1], 8, 8, 48), ([1000], 12, 4, 32), ([130, 129, 128], 16, 1, 64),
    ([40, 5], 40, 2, 24), ([33], 128, 1, 128), ([2000, 3], 6, 2, 256), ([17] * 30, 8, 2, 8), ([5000], 4, 1, 40),
]


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,hq,hkv,page", CASES)
def test_paged_attention_matches_the_definition(st, lens, hq, hkv, page, cache):
    rng = np.random.default_rng(sum(lens) + hq)
    a = _cache(rng, lens, hkv, page, cache)
    q = bf16(rng.normal(size=(len(lens), hq, 128)))
    o, err = _attend(st, a, q)
    assert err == [0, 0, 0, 0]
    _check(a, q, o)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_paged_attention_uneven_queries_and_scores(st, cache):
    """Rows of very large, very small and zero queries; scores that grow along the cache."""
    rng = np.random.default_rng(2)
    a = _cache(rng, [700, 90], 2, 16, cache)
    q = rng.normal(size=(2, 8, 128))
    q[:, 1] *= 20.0
    q[:, 2] *= 1e-6
    q[:, 3] = 0.0
    q[:, 4, :3] *= 300.0                       # a few strong channels
    o, err = _attend(st, a, bf16(q))
    assert err == [0, 0, 0, 0]
    _check(a, bf16(q), o)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_paged_attention_pages_out_of_range(st, cache):
    rng = np.random.default_rng(3)
    lens = [200, 300, 50]
    a = _cache(rng, lens, 2, 16, cache)
    q = bf16(rng.normal(size=(3, 8, 128)))
    a["table"][1, 7] = a["k_pages"].shape[0]
    o, err = _attend(st, a, q)
    assert err[:3] == [10, 1, 7]
    assert torch.all(o[1] == 7.0)
    _check(a, q, o, keep=(0, 2))
    a["table"][1, 7] = -1
    o, err = _attend(st, a, q)
    assert err[:3] == [10, 1, 7] and torch.all(o[1] == 7.0)


def test_paged_attention_lengths_are_clamped(st):
    rng = np.random.default_rng(4)
    a = _cache(rng, [64, 32], 1, 16, "bf16")
    a["table"] = a["table"][:, :4].contiguous()
    a["table"][1, 2:] = a["table"][0, :2]
    for n in ("k_pages", "v_pages"):
        a[n] = torch.nan_to_num(a[n])
    a["lens"] = i32([-3, 1000])
    q = bf16(rng.normal(size=(2, 4, 128)))
    o, err = _attend(st, a, q)
    assert err == [0, 0, 0, 0]
    assert torch.all(o[0] == 0)
    _check(a, q, o)


def test_paged_attention_in_graphs_that_share_a_workspace(st):
    rng = np.random.default_rng(5)
    size = st.stree_paged_attention_workspace_size(8, 2)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    runs = []
    for lens in ([900, 3], [40, 2000]):
        a = _cache(rng, lens, 2, 16, "bf16")
        q = bf16(rng.normal(size=(2, 8, 128)))
        want, _ = _attend(st, a, q)
        o = torch.zeros_like(q)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            st.stree_paged_attention(q, a["k_pages"], a["v_pages"], a["table"], a["lens"], o, SCALE, workspace=ws)
        runs.append((g, o, want, a, q))        # a graph's tensors live as long as the graph
    for _ in range(2):
        for g, *_ in runs:
            g.replay()
    torch.cuda.synchronize()
    for _, o, want, *_ in runs:
        assert torch.equal(o, want)            # the same order of sums every time


def test_paged_attention_workspace_too_small(st):
    rng = np.random.default_rng(6)
    a = _cache(rng, [5], 1, 8, "bf16")
    with pytest.raises(st.StreeError):
        _attend(st, a, bf16(rng.normal(size=(1, 4, 128))), workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))


def _empty_pages(n, hkv, page, cache):
    a = dict(k_scales=None, v_scales=None)
    for name in ("k", "v"):
        if cache == "bf16":
            a[name + "_pages"] = torch.full((n, hkv, page, 128), 3.0, dtype=torch.bfloat16, device="cuda")
        else:
            a[name + "_pages"] = torch.full((n, hkv, page, 128), 3.0, device="cuda").to(torch.float8_e4m3fn)
            a[name + "_scales"] = torch.full((n, hkv, page), 130, dtype=torch.uint8, device="cuda")
    return a


def _row(x, cache):
    """(scale byte, values) of a written row; bf16 pages keep the row."""
    return (130, x) if cache == "bf16" else oracle_cache_row(x)


def _expect(a, table, cache, writes):
    """The pages' values after `writes`: (sequence, position, rows of k and of v [H, 128])."""
    want = _values(a)
    scales = [None if a[n] is None else a[n].cpu().numpy().copy() for n in ("k_scales", "v_scales")]
    page = want[0].shape[2]
    for b, pos, *rows in writes:
        for x, w, s in zip(rows, want, scales):
            for h in range(x.shape[0]):
                byte, w[table[b, pos // page], h, pos % page] = _row(x[h], cache)
                if s is not None:
                    s[table[b, pos // page], h, pos % page] = byte
    return want, scales


def _same(a, want, scales):
    for n, w, s, x in zip(("k", "v"), want, scales, _values(a)):
        np.testing.assert_array_equal(x, w, err_msg=n)
        if s is not None:
            np.testing.assert_array_equal(a[n + "_scales"].cpu().numpy(), s, err_msg=n)


def _odd_rows(rng, n, hkv):
    """Rows of many sizes, zeros, a lone value, infinities and NaN, a scale's edge, bf16's largest."""
    x = rng.normal(size=(n, hkv, 128)) * np.exp(rng.normal(size=(n, hkv, 1)) * 4)
    flat = x.reshape(-1, 128)
    flat[0] = 0.0
    if len(flat) > 8:
        flat[1, 1:] = 0.0
        flat[2, :3] = [np.inf, -np.inf, np.nan]
        flat[3] = 448.0
        flat[4] = np.linspace(-450, 450, 128)
        flat[5] = 3.3895e38
        flat[6] *= 1e-38
        flat[7] = np.nan
    return bf16(x)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,start,hkv,page", [([1], [0], 1, 8), ([20, 0, 37], [5, 3, 90], 3, 16), ([130], [61], 2, 24),
                                                 ([1] * 17, list(range(17)), 4, 8)])
def test_cache_write_and_read(st, lens, start, hkv, page, cache):
    rng = np.random.default_rng(sum(lens) + page)
    ends = [s + n for s, n in zip(start, lens)]
    table, n_pages = random_tables(rng, ends, page)
    a = _empty_pages(n_pages, hkv, page, cache)
    extra = 2                                  # rows behind the last sequence
    k, v = _odd_rows(rng, sum(lens) + extra, hkv), _odd_rows(rng, sum(lens) + extra, hkv)
    at, writes = 0, []
    for b, n in enumerate(lens):
        writes += [(b, start[b] + i, f64(k[at + i]), f64(v[at + i])) for i in range(n)]
        at += n
    want, scales = _expect(a, table, cache, writes)
    err = torch.full((4,), -1, dtype=torch.int32, device="cuda")
    st.stree_cache_write(k, v, i32(offsets(lens)), i32(start), i32(table), a["k_pages"], a["v_pages"], k_scales=a["k_scales"],
                         v_scales=a["v_scales"], err_out=err)
    torch.cuda.synchronize()
    assert err.tolist() == [0, 0, 0, 0]
    _same(a, want, scales)
    cap = max(ends) + 3
    kc = torch.full((len(lens), cap, hkv, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    vc = torch.full_like(kc, 7.0)
    err.fill_(-1)
    st.stree_cache_read(a["k_pages"], a["v_pages"], i32(table), i32(ends), kc, vc, k_scales=a["k_scales"],
                        v_scales=a["v_scales"], err_out=err)
    torch.cuda.synchronize()
    assert err.tolist() == [0, 0, 0, 0]
    for got, w in ((kc, want[0]), (vc, want[1])):
        for b, n in enumerate(ends):
            np.testing.assert_array_equal(f64(got[b, :n]), oracle_pages(w, table[b], n))
            assert torch.all(got[b, n:] == 7.0)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_cache_commit_of_accepted_paths(st, cache):
    rng = np.random.default_rng(8)
    path = np.array([[0, 2, 5, -1], [0, -1, -1, -1], [3, 1, 4, 0], [9, 9, 9, 9]], np.int32)
    plen, start, page, hkv = [3, 0, 9, 1], [14, 7, 0, 30], 8, 2
    ends = [s + 4 for s in start]
    table, n_pages = random_tables(rng, ends, page)
    a = _empty_pages(n_pages, hkv, page, cache)
    k, v = _odd_rows(rng, 4 * 10, hkv).reshape(4, 10, hkv, 128), _odd_rows(rng, 4 * 10, hkv).reshape(4, 10, hkv, 128)
    writes = [(b, start[b] + i, f64(k[b, path[b, i]]), f64(v[b, path[b, i]])) for b in range(4) for i in range(min(plen[b], 4))]
    want, scales = _expect(a, table, cache, writes)
    err = torch.full((4,), -1, dtype=torch.int32, device="cuda")
    st.stree_cache_commit(k, v, i32(path), i32(plen), i32(start), i32(table), a["k_pages"], a["v_pages"],
                          k_scales=a["k_scales"], v_scales=a["v_scales"], err_out=err)
    torch.cuda.synchronize()
    assert err.tolist() == [0, 0, 0, 0]
    _same(a, want, scales)
    path[2, 1] = 10                            # no such node: that row alone is not written
    st.stree_cache_commit(k, v, i32(path), i32(plen), i32(start), i32(table), a["k_pages"], a["v_pages"],
                          k_scales=a["k_scales"], v_scales=a["v_scales"], err_out=err)
    torch.cuda.synchronize()
    assert err.tolist() == [4, 2, 1, 10]
    _same(a, want, scales)


def test_cache_write_refuses_what_does_not_fit(st):
    rng = np.random.default_rng(9)
    table = np.array([[0, 1], [2, 3], [4, BAD], [5, 6]], np.int32)
    a = _empty_pages(8, 1, 8, "bf16")
    lens, start = [10, 5, 12, 2], [7, 4, 0, -1]          # the first ends at 17 of 16, the last starts before 0
    k, v = bf16(rng.normal(size=(29, 1, 128))), bf16(rng.normal(size=(29, 1, 128)))
    writes = [(1, 4 + i, f64(k[10 + i]), f64(v[10 + i])) for i in range(5)]
    writes += [(2, i, f64(k[15 + i]), f64(v[15 + i])) for i in range(8)]   # the tokens on the page that exists
    want, scales = _expect(a, table, "bf16", writes)
    err = torch.full((4,), -1, dtype=torch.int32, device="cuda")
    st.stree_cache_write(k, v, i32(offsets(lens)), i32(start), i32(table), a["k_pages"], a["v_pages"], err_out=err)
    torch.cuda.synchronize()
    assert err[0] == 10 and int(err[1]) in (0, 2, 3)
    _same(a, want, scales)
    cu = i32([0, 10, 5, 27, 29])               # the second sequence's offsets go back
    st.stree_cache_write(k, v, cu, i32([0, 0, 0, 0]), i32(table[[0, 1, 3, 3]]), a["k_pages"], a["v_pages"], err_out=err)
    torch.cuda.synchronize()
    assert err[0] in (9, 10)


def test_cache_read_skips_pages_out_of_range(st):
    a = _empty_pages(4, 1, 8, "bf16")
    table = i32([[1, BAD, 2], [0, 1, 3]])
    kc = torch.full((2, 20, 1, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    vc = torch.full_like(kc, 7.0)
    err = torch.full((4,), -1, dtype=torch.int32, device="cuda")
    st.stree_cache_read(a["k_pages"], a["v_pages"], table, i32([24, 9]), kc, vc, err_out=err)
    torch.cuda.synchronize()
    assert err.tolist() == [10, 0, 1, BAD]
    assert torch.all(kc[0, :8] == 3) and torch.all(kc[0, 8:16] == 7) and torch.all(vc[0, 16:] == 3)
    assert torch.all(kc[1, :9] == 3) and torch.all(vc[1, 9:] == 7)


def test_binding_refuses_each_tensor(st):
    """Every tensor of a call in a wrong shape, dtype, order of memory or place."""
    rng = np.random.default_rng(10)
    a = _cache(rng, [20, 30], 2, 8, "e4m3")
    q = bf16(rng.normal(size=(2, 8, 128)))
    ws = torch.empty(st.stree_paged_attention_workspace_size(8, 2), dtype=torch.uint8, device="cuda")
    good = dict(q=q, k_pages=a["k_pages"], v_pages=a["v_pages"], page_table=a["table"], seq_len=a["lens"],
                o=torch.empty_like(q), scale=SCALE, k_scales=a["k_scales"], v_scales=a["v_scales"],
                err_out=torch.zeros(4, dtype=torch.int32, device="cuda"), workspace=ws)
    st.stree_paged_attention(**good)
    for name, t in good.items():
        if name == "scale":
            continue
        wrong = [t.cpu(), t.double() if t.dtype is not torch.float8_e4m3fn else t.view(torch.uint8)]
        if name not in ("workspace",):
            wrong.append(t[:-1])
        if t.dim() > 1:
            wrong.append(t.transpose(0, 1).contiguous().transpose(0, 1))
        for w in wrong:
            with pytest.raises((ValueError, TypeError)):
                st.stree_paged_attention(**{**good, name: w})
    with pytest.raises(ValueError):            # a key head count that the queries do not have
        st.stree_paged_attention(**{**good, "v_pages": a["v_pages"][:, :1].contiguous()})
    with pytest.raises(st.StreeError):
        st.stree_paged_attention(**{**good, "q": q[:, :7].contiguous(), "o": q[:, :7].contiguous()})


def test_offsets_beyond_32_bits(st):
    """Pages whose elements lie past 2^31 (and bytes past 2^32): written, attended over, read back."""
    n_pages, hkv, page = 36000, 8, 64              # 4.7 GB of bf16 keys, and of values
    kp = torch.empty((n_pages, hkv, page, 128), dtype=torch.bfloat16, device="cuda")
    vp = torch.empty_like(kp)
    table = i32([[n_pages - 1, 3, n_pages - 2], [n_pages - 3, 0, 0]])
    rng = np.random.default_rng(11)
    lens = [150, 40]
    k, v = bf16(rng.normal(size=(190, hkv, 128))), bf16(rng.normal(size=(190, hkv, 128)))
    st.stree_cache_write(k, v, i32(offsets(lens)), i32([0, 0]), table, kp, vp)
    kc = torch.empty((2, 150, hkv, 128), dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    st.stree_cache_read(kp, vp, table, i32(lens), kc, vc)
    torch.cuda.synchronize()
    assert torch.equal(kc[0], k[:150]) and torch.equal(vc[1, :40], v[150:])
    q = bf16(rng.normal(size=(2, 8, 128)))
    o, err = _attend(st, dict(k_pages=kp, v_pages=vp, k_scales=None, v_scales=None, table=table, lens=i32(lens)), q)
    assert err == [0, 0, 0, 0]
    for b, (lo, hi) in enumerate(((0, 150), (150, 190))):
        ref, oa = oracle_decode_attention(f64(q[b]), f64(k[lo:hi]), f64(v[lo:hi]), SCALE)
        within(f64(o[b]), ref, attention_tol(ref, oa, 40.0), f"sequence {b}")


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_paged_attention_many_sequences(st, cache):
    """More sequences than a block has threads, with empty ones among them."""
    rng = np.random.default_rng(12)
    lens = [int(n) for n in rng.integers(0, 20, size=700)]
    a = _cache(rng, lens, 1, 8, cache)
    q = bf16(rng.normal(size=(700, 4, 128)))
    o, err = _attend(st, a, q)
    assert err == [0, 0, 0, 0]
    _check(a, q, o)


def test_paged_attention_extreme_value_scales(st):
    """Rows of zeros (the least scale) beside rows of ordinary and of very large and small scales."""
    rng = np.random.default_rng(13)
    lens = [3000, 300, 90]
    a = _cache(rng, lens, 1, 16, "e4m3", stale=False)
    vs = a["v_scales"]
    vs.copy_(torch.from_numpy(rng.choice([100, 120, 140], size=tuple(vs.shape)).astype(np.uint8)))
    table = a["table"].cpu().numpy()
    for p in table[0, :100]:                       # most of the first sequence's values are zero rows
        a["v_pages"][p].zero_()
        vs[p] = 9
    for p in table[2, :6]:                         # all of the third's
        a["v_pages"][p].zero_()
        vs[p] = 9
    q = bf16(rng.normal(size=(3, 4, 128)))
    o, err = _attend(st, a, q)
    assert err == [0, 0, 0, 0]
    _check(a, q, o)
    assert torch.all(o[2] == 0)
