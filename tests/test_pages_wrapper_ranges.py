"""Numbers that the C entry points of the page lists and the selection cannot hold are refused by the wrappers: cut to 32 bits they
would be other, valid ones."""
import pytest

torch = pytest.importorskip("torch")

import flash_attention_backward_gb300 as fb  # noqa: E402
from flash_attention_backward_gb300 import build  # noqa: E402

WRAPS = 1 << 32


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def ints(*shape):
    return torch.zeros(shape, dtype=torch.int32)


@pytest.mark.parametrize("page_size", [WRAPS + 16, -WRAPS + 16, 1 << 31])
def test_a_page_size_beyond_32_bits_is_refused(page_size):
    with pytest.raises(fb.FaBackError, match="page_size"):
        fb.PageLists.empty(3, 2, 8, page_size, device="cpu")


@pytest.mark.parametrize("T", [WRAPS + 5, -1, 1 << 31])
def test_a_number_of_tokens_beyond_32_bits_is_refused(T):
    with pytest.raises(fb.FaBackError, match="T: "):
        fb.pages_extend(fb.PageLists.empty(3, 2, 8, 16, device="cpu"), ints(3), T)


@pytest.mark.parametrize("kw", [dict(K=WRAPS + 2), dict(first=WRAPS), dict(last=WRAPS + 1), dict(last=-WRAPS), dict(K=1 << 31), dict(first=-(1 << 31) - 1)])
def test_a_selection_beyond_32_bits_is_refused(kw):
    k = torch.zeros(4, 16, 2, fb.fa_row_bytes(fb.FA_Q8_0, 128), dtype=torch.uint8)
    cache = fb.PagedCache(k, fb.FA_Q8_0, k.clone(), fb.FA_Q8_0, ints(2, 2), D=128, Dv=128)
    with pytest.raises(fb.FaBackError, match="%s: " % list(kw)[0]):
        fb.page_select(torch.zeros(2, 4, 128), cache, fb.PageBounds.of(cache), ints(2), **{**dict(K=2, scale=1.0), **kw})


def test_tensors_beyond_32_bits_are_refused():
    def lists(B=3, width=2, n=8):
        t = [torch.empty(shape, dtype=torch.int32, device="meta") for shape in ((B, width), (B,), (n,), (1,))]
        return fb.PageLists(*t, page_size=16)
    assert lists().num_pages == 8
    for name, kw in (("free", dict(n=WRAPS + 8)), ("page_table", dict(width=WRAPS + 2)), ("page_table", dict(B=WRAPS + 3))):
        with pytest.raises(fb.FaBackError, match=name):
            lists(**kw)


def test_views_beyond_32_bits_are_refused():
    """(expanded: no memory behind them)"""
    x, rope, axes = torch.zeros(5, 2, 128), fb.rope_frequencies(64, device="cpu"), fb.rope_sections([16, 16], device="cpu")
    with pytest.raises(fb.FaBackError, match="pos: "):
        fb.qk_norm_rope(x, None, ints(1, 5).expand(WRAPS + 2, 5), rope=rope, rope_axes=axes)
    k = torch.zeros(4, 16, 2, fb.fa_row_bytes(fb.FA_Q8_0, 128), dtype=torch.uint8)
    cache = fb.PagedCache(k, fb.FA_Q8_0, k.clone(), fb.FA_Q8_0, ints(2, 2), D=128, Dv=128)
    with pytest.raises(fb.FaBackError, match="pages: "):
        fb.paged_decode(torch.zeros(2, 4, 128), cache, ints(2), scale=1.0, pages=torch.empty(2, 2, WRAPS + 4, dtype=torch.int32, device="meta"))
