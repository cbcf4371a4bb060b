"""8-bit pages: scores and weights far apart in size (a key that takes nearly all of the softmax, channels of a
query next to much stronger ones) keep their precision."""
import numpy as np
import pytest
import torch

from oracle.prompt import oracle_decode_attention

from prompt_util import attention_tol, bf16, f64, i32, within

pytestmark = pytest.mark.gpu
SCALE = 0.09
PAGE = 16


@pytest.fixture(scope="module")
def st():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from hybrid_packed_tree_b200 import stree
    return stree


def _run(st, q, k, v, k_scale, v_scale):
    """One sequence over one key/value head: q [Hq, 128], k, v [n, 128] as e4m3 elements, scale bytes [n]."""
    n = k.shape[0]
    pages = -(-n // PAGE)
    fill = pages * PAGE - n

    def paged(x, s):
        x = np.concatenate([x, np.full((fill, 128), np.nan)]).reshape(pages, 1, PAGE, 128)
        s = np.concatenate([s, np.full(fill, 255)]).reshape(pages, 1, PAGE)
        e = torch.from_numpy(x.astype(np.float32)).to(torch.float8_e4m3fn)
        return e.cuda(), torch.from_numpy(s.astype(np.uint8)).cuda(), e.double().numpy().reshape(-1, 128)[:n] * 2.0 ** (s.reshape(-1)[:n, None] - 127.0)

    kp, ks, kx = paged(k, k_scale)
    vp, vs, vx = paged(v, v_scale)
    qd = bf16(q[None])
    o = torch.full_like(qd, 7.0)
    err = torch.full((4,), -1, dtype=torch.int32, device="cuda")
    ws = torch.full((st.stree_paged_attention_workspace_size(q.shape[0], 1),), 0xFF, dtype=torch.uint8, device="cuda")
    st.stree_paged_attention(qd, kp, vp, i32(np.arange(pages)[None]), i32([n]), o, SCALE, k_scales=ks, v_scales=vs, err_out=err,
                             workspace=ws)
    torch.cuda.synchronize()
    assert err.tolist() == [0, 0, 0, 0]
    ref, oa = oracle_decode_attention(f64(qd[0]), kx[:, None], vx[:, None], SCALE)
    score = SCALE * np.max(np.abs(f64(qd[0])) @ np.abs(kx).T)
    within(f64(o[0]), ref, attention_tol(ref, oa, score), "output")


@pytest.mark.parametrize("hq", [4, 12])
@pytest.mark.parametrize("strong", [1.25, 1.625, 1.75])
@pytest.mark.parametrize("n", [40, 3000])
def test_weights_beside_a_key_that_takes_nearly_all(st, n, strong, hq):
    """The strong key's value is zero, so the output is what the others hold: weights of 2^-21 to 2^-29 each."""
    rng = np.random.default_rng(n)
    k, v = np.zeros((n, 128)), np.abs(rng.normal(size=(n, 128))) + 0.5
    k[n // 3], v[n // 3] = strong, 0.0
    _run(st, np.ones((hq, 128)), k, v, np.full(n, 127), np.full(n, 127))


@pytest.mark.parametrize("hq", [4, 12])
@pytest.mark.parametrize("weak", [2.0 ** -12, 2.0 ** -20, 2.0 ** -26])
def test_channels_of_a_query_beside_a_strong_one(st, weak, hq):
    """Keys that are zero where the query is strong: the weak channels decide the scores."""
    rng = np.random.default_rng(5)
    n = 300
    q = weak * rng.uniform(1.0, 2.0, size=(hq, 128))
    q[:, 0] = 1.0
    k = rng.normal(size=(n, 128)) * 100
    k[:, 0] = 0.0
    _run(st, q, k, rng.normal(size=(n, 128)), np.full(n, 127 - 5 - int(np.log2(weak))), rng.integers(119, 130, size=n))


def test_the_smallest_and_largest_scales(st):
    """Value rows of every size that a scale can hold, and a query of zeros and of very small elements."""
    rng = np.random.default_rng(6)
    n = 64
    for byte in (9, 24, 127, 230, 246):
        q = rng.normal(size=(3, 128))
        q[1] = 0.0
        q[2] *= 2.0 ** -120
        _run(st, q, rng.normal(size=(n, 128)), rng.normal(size=(n, 128)), np.full(n, 127), np.full(n, byte))
