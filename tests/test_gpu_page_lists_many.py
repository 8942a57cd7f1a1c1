"""Page lists of more requests than a CTA holds the starts of (8192), on the GPU, against lists."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_paged_ext import cuda, fb, lists_of, same_lists  # noqa: E402,F401


@pytest.mark.parametrize("B, tokens, behind", [(8192, 6, 3), (8193, 6, 0), (20000, 2, 9001), (9000, 1, 0)])
def test_extend_and_trim_of_many_requests(fb, B, tokens, behind):
    """Some find no pages and some no room; `behind` tokens of T belong to nobody; then T ends inside the requests."""
    rng = np.random.default_rng(B)
    lists, ref = lists_of(fb, rng, B, 3, 2 * B, 4, 0.6)
    for step in range(3):
        news = np.where(rng.random(B) < 0.2, rng.integers(-2, 1, B), rng.integers(1, tokens + 1, B)).astype(np.int32)
        need = int(np.maximum(news, 0)[np.array(ref.lens) >= 0].sum())
        T = need + behind if step < 2 else need - need // 10 - 1
        got, want = fb.pages_extend(lists, cuda(news), T), ref.extend(news.tolist(), T)
        for n, x in want.items():
            assert got[n].tolist() == x, (step, n)
        same_lists(lists, ref)
        keep = np.where(rng.random(B) < 0.5, -1, rng.integers(0, 13, B)).astype(np.int32)
        fb.pages_trim(lists, cuda(keep))
        ref.trim(keep.tolist())
        same_lists(lists, ref)
    assert fb.fa_back_get_error() == 0
