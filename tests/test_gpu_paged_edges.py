"""The paged-cache and norm / rotation operators at their edges: the error word, orders on a stream, values that
are not finite, the ends of the types' ranges, and how near f32 outputs are to 64 bits."""
import numpy as np
import pytest

import paged_ref as R
from test_gpu_paged import F16, F32, Q4, Q8, U, act_array, check_decode, cuda, empty_cache, fb, within  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def test_a_page_report_does_not_hide_a_timeout(fb):
    """After a timeout the outputs are undefined, after an invalid page they are not: the timeout is what stays,
    whichever comes first."""
    p = R.Paged(8, [700, 90], 2, 64, 64, Q8, Q8, 16)
    q, cache, out = check_decode(fb, p, 4)
    lens = cuda(np.array(p.lens, np.int32))
    x, one = torch.ones(1, 2, 64, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")

    def bad_page():
        fb.cache_append(x, x, cache, one * 5, one)  # no such sequence

    def bad_length():
        fb.paged_decode(q, cache, lens + 10 ** 6, scale=0.125)

    def timeout():
        assert fb.fa_back_test_wait_limit(0) == 0
        fb.paged_decode(q, cache, lens, scale=0.125)

    for calls, want in (((timeout, bad_page), "FA_ERR_TIMEOUT"), ((bad_page, timeout), "FA_ERR_TIMEOUT"),
                        ((timeout, bad_length), "FA_ERR_TIMEOUT"), ((bad_page, bad_length), "FA_ERR_PAGE")):
        for c in calls:
            c()
        assert fb.STATUS[fb.fa_back_get_error()] == want
        assert fb.fa_back_get_error() == 0


def test_lengths_and_pages_written_just_before(fb):
    """Each call sees the lengths, positions and page numbers that the kernel before it on the stream has written."""
    p = R.Paged(9, [3000, 40, 900], 2, 64, 64, Q8, F16, 16)
    q, cache, _ = check_decode(fb, p, 4)
    full, table = cuda(np.array(p.lens, np.int32)), cache.page_table.clone()
    steps = [full - 30 * i for i in range(1, 30)]
    kw = dict(scale=0.125)
    want = []
    for n in steps:
        cache.page_table.copy_(table if len(want) % 2 else table.flip(1))
        n = n.clamp(min=1)
        torch.cuda.synchronize()
        want.append(fb.paged_decode(q, cache, n, **kw))
        torch.cuda.synchronize()
    lens, got = torch.zeros_like(full), []
    pos, seq = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    rows = torch.cat([fb.cache_read(cache, seq, seq + j, dtype=torch.uint8)["k"] for j in range(40)])
    for _ in range(5):
        for i, n in enumerate(steps):
            torch.clamp(n, min=1, out=lens)
            cache.page_table.copy_(table if i % 2 else table.flip(1))
            got.append(fb.paged_decode(q, cache, lens, **kw))
    for i, g in enumerate(got):
        w = want[i % len(steps)]
        for n in ("O", "lse"):  # bits: with the flipped table short sequences' pages have rows of NaN
            assert torch.equal(g[n].view(torch.int32), w[n].view(torch.int32))
            assert i % len(steps) % 2 == 0 or bool(torch.isfinite(g[n]).all())
    cache.page_table.copy_(table if (len(steps) - 1) % 2 else table.flip(1))
    for j in range(40):  # reads that follow a position counted up on the device
        g = fb.cache_read(cache, seq, pos, dtype=torch.uint8)["k"]
        pos.add_(1)
        assert torch.equal(g[0], rows[j])
    fb.fa_back_get_error()  # (the flipped table's unused pages)
