"""A decay of zero forgets: what a state held before it leaves no trace, however large it was."""
import numpy as np
import pytest
import torch

from prompt_util import bf16, f32, i32, offsets

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def st():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from hybrid_packed_tree_b200 import stree
    return stree


@pytest.mark.parametrize("lens,dv,dtype", [([3], 128, "bf16"), ([128], 64, "bf16"), ([129, 300], 128, "bf16"),
                                           ([2300, 1900], 128, "bf16"), ([40], 64, "f32")])
def test_decay_of_zero_leaves_nothing(st, lens, dv, dtype):
    """Only the tokens up to the zero have keys and values; the state and every later output are exactly zero."""
    rng = np.random.default_rng(sum(lens))
    n, b, hv, hk = sum(lens), len(lens), 2, 1
    up = bf16 if dtype == "bf16" else f32
    q, k, v = up(rng.normal(size=(n, hk, 128))), up(rng.normal(size=(n, hk, 128))), up(rng.normal(size=(n, hv, dv)))
    alpha, beta = np.full((n, hv), 0.999), np.zeros((n, hv))
    at = offsets(lens)
    for lo, hi in zip(at, at[1:]):             # the last zero: in the first chunk, and where there are several in the last
        for zero in (lo + 1, hi - 2):
            alpha[zero] = 0.0
        beta[lo:hi - 2] = 1e30                 # before the zero alone
    S0 = f32(rng.normal(0, 1e30, size=(b, hv, dv, 128)))
    o, S = torch.full_like(v, 7.0), torch.full_like(S0, 7.0)
    ws = torch.full((max(16, st.stree_linear_prompt_workspace_size(b, n, hv, hk, 128, dv, v.dtype)),), 0xFF, dtype=torch.uint8, device="cuda")
    st.stree_linear_prompt(q, k, v, f32(alpha), f32(beta), i32(at), o, S0=S0, S_new=S, workspace=ws)
    torch.cuda.synchronize()
    assert torch.all(S == 0), S.abs().max().item()
    for hi in at[1:]:
        assert torch.all(o[hi - 2:hi] == 0), o[hi - 2:hi].abs().max().item()


@pytest.mark.parametrize("dv", [128, 64])
def test_small_decays_are_not_zero(st, dv):
    """Decays down to the smallest float keep what they keep."""
    tiny = np.array([2.0 ** -100, 2.0 ** -125, 2.0 ** -127, 2.0 ** -140, 2.0 ** -149])
    b = len(tiny)
    rng = np.random.default_rng(3)
    S0 = f32(rng.choice([-1.0, 1.0], size=(b, 2, dv, 128)) * 2.0 ** 120)
    zero = torch.zeros((b, 1, 128), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros((b, 2, dv), dtype=torch.bfloat16, device="cuda")
    alpha = torch.from_numpy(np.repeat(tiny[:, None], 2, 1).astype(np.float32)).cuda()
    o, S = torch.empty_like(v), torch.empty_like(S0)
    st.stree_linear_prompt(zero, zero, v, alpha, None, i32(np.arange(b + 1)), o, S0=S0, S_new=S)
    torch.cuda.synchronize()
    want = S0.double() * torch.from_numpy(tiny).cuda()[:, None, None, None]
    # The logarithm's rounding (half a step of at most 149, 2^-17) twice, 2^x within 2^-22, and a decay below
    # the normal numbers is rounded to a multiple of 2^-149.
    bound = want.abs() * 2.0 ** -15 + 2.0 ** -150 * S0.double().abs()
    assert torch.all((S.double() - want).abs() <= bound)
