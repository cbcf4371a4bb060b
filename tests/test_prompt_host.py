"""Refusals of the prompt, single-token and cache calls: shapes, dtypes, pointers and
alignment are checked on the host before any device work, and the binding checks shapes
and devices of its tensors."""
import ctypes

import pytest
import torch

OK = 0x10000                                   # aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    from hybrid_packed_tree_b200.build import build
    build()
    from hybrid_packed_tree_b200 import stree
    return stree._lib


def _call(fn, args, **over):
    a = list(args)
    for i, v in over.items():
        a[int(i[1:])] = v
    return fn(*a)


def test_linear_prompt(lib):
    # q k v alpha beta skip S0 cu; total batch Hv Hk dk dv dtype; o S_new ws bytes err stream
    base = [OK] * 8 + [64, 2, 8, 4, 128, 128, 1] + [OK, OK, None, 0, None, None]
    fn = lib.stree_linear_prompt
    for over in (dict(i8=-1), dict(i9=-1), dict(i11=3), dict(i11=0), dict(i12=4), dict(i12=264), dict(i12=12), dict(i13=0),
                 dict(i13=257), dict(i14=2), dict(i14=7)):
        assert _call(fn, base, **over) == 2, over
    for i in (0, 1, 2, 3, 7, 15):
        assert _call(fn, base, **{f"i{i}": None}) == 1, i
    for i in (0, 1, 2, 6, 15, 16):
        assert _call(fn, base, **{f"i{i}": OK + 8}) == 5, i
    assert _call(fn, base, i3=OK + 2) == 5
    assert _call(fn, base, i17=OK + 8, i18=64) == 5
    assert _call(fn, base, i9=0) == 0          # no sequence: nothing to do
    size = ctypes.c_size_t(7)
    assert lib.stree_linear_prompt_workspace_size(1, 64, 8, 3, 128, 128, 1, ctypes.byref(size)) == 2
    assert lib.stree_linear_prompt_workspace_size(1, 64, 8, 4, 128, 128, 1, None) == 1


def test_linear_step(lib):
    # q k v alpha beta skip S0; batch Hv Hk dk dv dtype; o S_new stream
    base = [OK] * 7 + [2, 8, 4, 128, 64, 0] + [OK, OK, None]
    fn = lib.stree_linear_step
    for over in (dict(i7=-1), dict(i9=3), dict(i10=130), dict(i11=12), dict(i12=2)):
        assert _call(fn, base, **over) == 2, over
    for i in (0, 1, 2, 3, 6, 13, 14):
        assert _call(fn, base, **{f"i{i}": None}) == 1, i
    for i in (0, 6, 13, 14):
        assert _call(fn, base, **{f"i{i}": OK + 4}) == 5, i
    assert _call(fn, base, i7=0) == 0


def test_prompt_attention(lib):
    # q k v cu; total batch Hq Hkv d; scale dtype o err stream
    base = [OK] * 4 + [64, 2, 32, 8, 128, 0.1, 1, OK, None, None]
    fn = lib.stree_prompt_attention
    for over in (dict(i4=-1), dict(i5=-1), dict(i7=5), dict(i7=0), dict(i6=129, i7=1), dict(i8=64), dict(i10=0), dict(i10=2)):
        assert _call(fn, base, **over) == 2, over
    for over in (dict(i9=0.0), dict(i9=-1.0), dict(i9=float("nan")), dict(i0=None), dict(i3=None), dict(i11=None)):
        assert _call(fn, base, **over) == 1, over
    for over in (dict(i0=OK + 8), dict(i1=OK + 2), dict(i11=OK + 4), dict(i3=OK + 1), dict(i12=OK + 2)):
        assert _call(fn, base, **over) == 5, over
    assert _call(fn, base, i5=0) == 0


PAGES = [16, 64, 4]                            # n_pages, page size, pages per sequence


def test_paged_attention(lib):
    # q kp vp ks vs table lens; batch Hq Hkv d pages..; scale dtype cache o ws bytes err stream
    base = [OK] * 3 + [None, None, OK, OK] + [2, 32, 8, 128] + PAGES + [0.1, 1, 1, OK, OK, 1 << 26, None, None]
    fn = lib.stree_paged_attention
    for over in (dict(i7=-1), dict(i9=5), dict(i10=64), dict(i11=0), dict(i12=4), dict(i12=12), dict(i12=8192), dict(i13=0),
                 dict(i15=0), dict(i16=0), dict(i16=5), dict(i11=1 << 28), dict(i13=1 << 27)):
        assert _call(fn, base, **over) == 2, over
    for over in (dict(i14=0.0), dict(i0=None), dict(i1=None), dict(i2=None), dict(i5=None), dict(i6=None), dict(i17=None),
                 dict(i18=None), dict(i3=OK), dict(i16=2), dict(i16=2, i3=OK)):
        assert _call(fn, base, **over) == 1, over
    for over in (dict(i0=OK + 8), dict(i1=OK + 8), dict(i17=OK + 2), dict(i18=OK + 8), dict(i6=OK + 1),
                 dict(i16=2, i3=OK + 8, i4=OK)):
        assert _call(fn, base, **over) == 5, over
    assert _call(fn, base, i7=0) == 0
    assert lib.stree_paged_attention_workspace_size(32, 5, 128, ctypes.byref(ctypes.c_size_t())) == 2
    assert lib.stree_paged_attention_workspace_size(32, 8, 64, ctypes.byref(ctypes.c_size_t())) == 2


def test_cache_calls(lib):
    # k v cu start table; total batch H d pages..; dtype cache kp vp ks vs err stream
    write = [OK] * 5 + [64, 2, 8, 128] + PAGES + [1, 1, OK, OK, None, None, None, None]
    for over in (dict(i5=-1), dict(i6=-1), dict(i7=0), dict(i8=96), dict(i10=7), dict(i12=0), dict(i13=0), dict(i13=3)):
        assert _call(lib.stree_cache_write, write, **over) == 2, over
    for over in (dict(i0=None), dict(i2=None), dict(i3=None), dict(i4=None), dict(i14=None), dict(i16=OK), dict(i13=2)):
        assert _call(lib.stree_cache_write, write, **over) == 1, over
    for over in (dict(i0=OK + 8), dict(i14=OK + 8), dict(i3=OK + 2), dict(i13=2, i16=OK, i17=OK + 4)):
        assert _call(lib.stree_cache_write, write, **over) == 5, over
    assert _call(lib.stree_cache_write, write, i6=0) == 0
    # k v path len maxlen start table; T batch H d pages..; dtype cache kp vp ks vs err stream
    commit = [OK] * 4 + [5, OK, OK] + [26, 2, 8, 128] + PAGES + [1, 1, OK, OK, None, None, None, None]
    for over in (dict(i4=0), dict(i4=257), dict(i7=0), dict(i7=257), dict(i8=-1), dict(i14=0)):
        assert _call(lib.stree_cache_commit, commit, **over) == 2, over
    for over in (dict(i0=None), dict(i2=None), dict(i3=None), dict(i5=None), dict(i6=None), dict(i17=None)):
        assert _call(lib.stree_cache_commit, commit, **over) == 1, over
    assert _call(lib.stree_cache_commit, commit, i1=OK + 8) == 5
    assert _call(lib.stree_cache_commit, commit, i8=0) == 0
    # kp vp ks vs table lens; batch S H d pages..; cache dtype kc vc err stream
    read = [OK, OK, None, None, OK, OK] + [2, 256, 8, 128] + PAGES + [1, 1, OK, OK, None, None]
    for over in (dict(i7=-1), dict(i9=64), dict(i13=0), dict(i14=2)):
        assert _call(lib.stree_cache_read, read, **over) == 2, over
    for over in (dict(i0=None), dict(i4=None), dict(i5=None), dict(i15=None), dict(i2=OK)):
        assert _call(lib.stree_cache_read, read, **over) == 1, over
    assert _call(lib.stree_cache_read, read, i16=OK + 8) == 5
    assert _call(lib.stree_cache_read, read, i6=0) == 0


def test_binding_refuses_on_the_host(lib):
    """No call reaches the library with tensors of other shapes, dtypes or devices."""
    from hybrid_packed_tree_b200 import stree
    bf = dict(dtype=torch.bfloat16)
    q, k = torch.zeros(5, 4, 128, **bf), torch.zeros(5, 2, 128, **bf)
    cu = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        stree.stree_prompt_attention(q, k, k, cu, q, 0.1)
    with pytest.raises(ValueError, match="q has shape"):
        stree.stree_linear_prompt(k[:4], k, q, torch.zeros(5, 4), None, cu, q)
    with pytest.raises(TypeError, match="q has dtype"):
        stree.stree_linear_step(k.float(), k, q, torch.zeros(5, 4), None, torch.zeros(5, 4, 128, 128), q, torch.zeros(5, 4, 128, 128))
    with pytest.raises(TypeError, match="q must be a torch.Tensor"):
        stree.stree_linear_prompt(None, k, q, torch.zeros(5, 4), None, cu, q)
    pages = torch.zeros(3, 2, 16, 128, **bf)
    table = torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="k_pages must be a CUDA tensor"):
        stree.stree_cache_write(k, k, cu, table[:, 0], table, pages, pages)
    with pytest.raises(ValueError, match="go with float8"):
        stree.stree_cache_write(k, k, cu, table[:, 0], table, pages, pages, k_scales=torch.zeros(3, 2, 16, dtype=torch.uint8))
    with pytest.raises(ValueError, match="go with float8"):
        stree.stree_cache_read(pages.to(torch.float8_e4m3fn), pages, table, cu[:2], pages[:2], pages[:2])
    with pytest.raises(TypeError, match="expected torch.bfloat16 or torch.float8_e4m3fn"):
        stree.stree_paged_attention(q[:2], pages.float(), pages, table, cu[:2], q[:2], 0.1)
    with pytest.raises(ValueError, match="page_table"):
        stree.stree_paged_attention(q[:2], pages, pages, table[0], cu[:2], q[:2], 0.1)
