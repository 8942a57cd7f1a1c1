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
