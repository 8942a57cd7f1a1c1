"""Bounds of quantised keys whose block scales are not finite, on the GPU."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_paged_ext import cuda, fb  # noqa: E402,F401


@pytest.mark.parametrize("name, codes", [("q8_0", 0), ("q8_0", 5), ("q4_0", 0x88), ("q4_0", 0x3a)])
@pytest.mark.parametrize("rows", [1, 9, 40])
def test_blocks_without_a_finite_scale(fb, name, codes, rows):
    """Page 0: an infinite scale in the first block of the last row, page 1: a NaN; the second block is finite in both."""
    t, rb = (fb.FA_Q8_0, 68) if name == "q8_0" else (fb.FA_Q4_0, 36)
    k = np.zeros((2, 64, 1, rb), np.uint8)
    for page, bad in ((0, np.inf), (1, np.nan)):
        k[page, :rows, 0, rb // 2:rb // 2 + 2] = np.frombuffer(np.float16(0.5).tobytes(), np.uint8)
        k[page, :rows, 0, rb // 2 + 2:] = 2 if t == fb.FA_Q8_0 else 0xaa  # 2 x 0.5
        k[page, :rows, 0, 2:rb // 2] = codes
        k[page, :rows, 0, :2] = np.frombuffer(np.float16(0.25).tobytes(), np.uint8)
        k[page, rows - 1, 0, :2] = np.frombuffer(np.float16(bad).tobytes(), np.uint8)
    cache = fb.PagedCache(cuda(k), t, cuda(k), t, cuda(np.array([[0, -1], [1, -1]], np.int32)), D=64, Dv=64)
    bounds = fb.PageBounds.of(cache)
    fb.page_bounds(cache, bounds, cuda(np.array([rows, rows], np.int32)))
    c, s = bounds.codes[:, 0].cpu().numpy(), bounds.scales[:, 0].cpu().numpy()
    assert s[0, 0] == np.inf and (c[0, 0, :32] == 127).all() and (c[0, 1, :32] == -127).all()
    if rows == 1:  # nothing but NaN
        assert s[1, 0] == np.inf and (c[1, 0, :32] == 127).all() and (c[1, 1, :32] == -127).all()
    else:  # a NaN is left out: the other rows' values
        v = 0.25 * np.array([codes] * 32 if t == fb.FA_Q8_0 else [(codes & 15) - 8] * 16 + [(codes >> 4) - 8] * 16, np.float32)
        top = np.abs(v).max()
        assert s[1, 0] == np.float32(top) / np.float32(127)
        if top:
            x = v / s[1, 0]
            assert (c[1, 0, :32] == np.ceil(x).clip(-127, 127)).all() and (c[1, 1, :32] == np.floor(x).clip(-127, 127)).all()
    assert (s[:, 1] == np.float32(1) / np.float32(127)).all() and (c[:, :, 32:] == 127).all()
    assert fb.fa_back_get_error() == 0
