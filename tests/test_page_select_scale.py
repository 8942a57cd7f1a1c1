"""The scale that page selection takes, on the host: one that is not finite orders nothing."""
import pytest

torch = pytest.importorskip("torch")

import flash_attention_backward_gb300 as fb  # noqa: E402
from flash_attention_backward_gb300 import build  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


@pytest.mark.parametrize("scale", [float("nan"), float("inf"), -float("inf")])
def test_a_scale_that_is_not_finite_is_refused(scale):
    cache = fb.fa_paged_cache(k=0x10000, v=0x20000, page_table=0x30000, k_type=2, v_type=2, num_pages=8, page_size=16, B=2, max_pages=4,
                              Hkv=2, D=128, Dv=128)
    rc = fb.fa_page_select(q=0x40000, act=0, q_row=1024, q_head=128, cache=cache, bounds=fb.fa_page_bounds_pool(0x100000, 0x200000),
                           seq_lens=0x50000, H=8, scale=scale, alibi_slopes=None, K=3, first=1, last=1, pages=0x300000,
                           workspace=0x400000, workspace_bytes=1 << 30, stream=None)
    assert fb.STATUS[rc] == "FA_ERR_SHAPE"
