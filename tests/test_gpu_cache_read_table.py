"""Reading more positions than a page table holds is reported, as writing them is."""
import pytest
import torch

from prompt_util import i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_cache_read_past_the_table_is_reported(cache):
    from hybrid_packed_tree_b200 import stree as st
    pages = torch.full((4, 1, 8, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    scales = None
    if cache == "e4m3":
        pages, scales = pages.float().to(torch.float8_e4m3fn), torch.full((4, 1, 8), 127, dtype=torch.uint8, device="cuda")
    table = i32([[0, 1], [2, 3]])              # 16 positions each
    kc = torch.full((2, 40, 1, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    vc = torch.full_like(kc, 7.0)
    err = torch.full((4,), -1, dtype=torch.int32, device="cuda")

    def read(lens, k, v):
        st.stree_cache_read(pages, pages, table, i32(lens), k, v, k_scales=scales, v_scales=scales, err_out=err)
        torch.cuda.synchronize()
        return err.tolist()

    assert read([16, 17], kc, vc) == [10, 1, 0, 17]
    for c in (kc, vc):
        assert torch.all(c[:, :16] == 3) and torch.all(c[:, 16:] == 7)   # what the table holds has been read
    assert read([16, 0], kc, vc) == [0, 0, 0, 0]
    # What the contiguous cache does not hold is not asked of the table.
    assert read([100, 100], kc[:, :16].contiguous(), vc[:, :16].contiguous()) == [0, 0, 0, 0]
    assert read([100, -5], kc, vc) == [10, 0, 0, 40]
