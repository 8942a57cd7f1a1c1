"""The operators around the paged cache on the GPU: keys stored through either path, positions of several axes,
page lists, page bounds, page selection and attention over selected pages, against 64-bit numpy.

Tolerances are bounds from the roundings that each operator makes, written beside them; whole numbers are equal.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def fb():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import flash_attention_backward_gb300 as m
    from flash_attention_backward_gb300 import build
    build.build()
    return m


def cuda(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def empty_cache(fb, B, max_pages, page, Hkv, D, Dv, kt, vt, seed=0):
    n = B * max_pages + 2
    table = np.random.default_rng(seed).permutation(n)[: B * max_pages].reshape(B, max_pages).astype(np.int32)
    k = torch.zeros((n, page, Hkv, fb.fa_row_bytes(kt, D)), dtype=torch.uint8, device="cuda")
    v = torch.zeros((n, page, Hkv, fb.fa_row_bytes(vt, Dv)), dtype=torch.uint8, device="cuda")
    return fb.PagedCache(k, kt, v, vt, cuda(table), D=D, Dv=Dv)


# ------------------------------------------------------------------------------------------------
# keys normalised and rotated on the way into the cache, or beforehand

@pytest.mark.parametrize("D, n_rot, halves, view", [
    (64, 64, True, False), (64, 32, True, True), (128, 128, True, False), (128, 0, True, False), (128, 128, False, False),
    (256, 256, True, False), (256, 64, True, True), (256, 34, False, True)])
def test_keys_are_the_same_bits_through_either_path(fb, D, n_rot, halves, view):
    """cache_append() with a norm and a rotation stores what qk_norm_rope() and a plain cache_append() store: the same
    sums in the same order.  f32 rows show every bit; 9000 rows of each."""
    gen = torch.Generator(device="cuda").manual_seed(D + n_rot)
    T, Hkv = 3000, 3
    x = torch.randn(T, 2 * Hkv + view, D + view, generator=gen, device="cuda")[..., :D]  # (a view: rows off 16 bytes)
    xk, xv = x[:, :Hkv], x[:, Hkv:2 * Hkv]
    w = 0.5 + torch.rand(D, generator=gen, device="cuda")
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    seq = torch.zeros_like(pos)
    rope, style = fb.rope_frequencies(n_rot) if n_rot else None, int(halves)
    y = fb.qk_norm_rope(xk, None, pos, wq=w, rope=rope, rope_style=style)["q"]
    one, two = (empty_cache(fb, 1, -(-T // 16), 16, Hkv, D, D, fb.FA_F32, fb.FA_Q8_0) for _ in range(2))
    fb.cache_append(xk, xv, one, seq, pos, k_norm=w, rope=rope, rope_style=style)
    fb.cache_append(y, xv, two, seq, pos)
    assert torch.equal(one.k, two.k) and torch.equal(one.v, two.v)
    assert fb.fa_back_get_error() == 0
