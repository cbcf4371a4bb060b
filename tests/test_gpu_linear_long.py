"""Long linear prompts against the definition: every number of segments up to the nine of a split, segments
without a chunk in the same call, and the walk on the CUDA cores at some thousand tokens."""
import numpy as np
import pytest
import torch

from test_gpu_linear import _check, _inputs, _run

pytestmark = pytest.mark.gpu
STATE = 128 * 128 * 4 + 32                     # workspace bytes of an item's segment


@pytest.fixture(scope="module")
def st():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from hybrid_packed_tree_b200 import stree
    return stree


@pytest.mark.parametrize("dv", [128, 64])
@pytest.mark.parametrize("total", [1024, 1536, 2048, 2560, 3100, 3584, 4096, 5000])
def test_every_number_of_segments(st, total, dv):
    hv = 128 // dv
    a = _inputs([total], hv, 1, 128, dv, "bf16", seed=total, decay=np.full(hv, 2e-3))
    segments = min(9, total // 512 + 1)
    assert st.stree_linear_prompt_workspace_size(1, total, hv, 1, 128, dv) == (segments - 1) * STATE
    o, S, err = _run(st, a)
    assert err == [0, 0, 0, 0]
    _check(a, o, S, f"{segments} segments")


@pytest.mark.parametrize("dv", [128, 64])
@pytest.mark.parametrize("lens,segments", [([8300, 1], 9), ([8300, 1, 0, 700], 5)])
def test_splits_of_uneven_sequences(st, lens, segments, dv):
    hv = 256 // dv
    a = _inputs(lens, hv, 1, 128, dv, "bf16", seed=dv, decay=np.geomspace(1e-3, 0.1, hv))
    assert st.stree_linear_prompt_workspace_size(len(lens), sum(lens), hv, 1, 128, dv) == 2 * len(lens) * (segments - 1) * STATE
    o, S, err = _run(st, a)
    assert err == [0, 0, 0, 0]
    _check(a, o, S, "uneven sequences")


def test_long_walks_on_the_cuda_cores(st):
    for shape in (([4100], 2, 1, 64, 32, "f32"), ([2000, 1], 3, 1, 128, 96, "bf16")):
        a = _inputs(*shape, seed=4, decay=np.full(shape[1], 1e-3))
        o, S, err = _run(st, a)
        assert err == [0, 0, 0, 0]
        _check(a, o, S, "walk")
