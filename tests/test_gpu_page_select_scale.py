"""Page selection with negative scales on the GPU: the pages whose bounds promise the largest scores, as with positive ones."""
import numpy as np
import pytest

import paged_ext_ref as E
import paged_ref as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_paged_ext import act_array, bounded_cache, cuda, fb  # noqa: E402,F401


@pytest.mark.parametrize("n, D, Hkv, G, act, slopes", [(700, 64, 1, 3, "f32", False), (90, 128, 2, 9, "bf16", True), (1500, 256, 1, 2, "f16", True),
                                                       (45000, 64, 1, 2, "f32", False)])
def test_a_negative_scale_counts_as_its_magnitude_of_the_other_query(fb, n, D, Hkv, G, act, slopes):
    """scale q.k = |scale| (-q).k, and so are the bounds of it."""
    rng = np.random.default_rng(n)
    cache, bounds, codes, scales, table = bounded_cache(fb, rng, n, D, Hkv, 1)
    q, qa = act_array(rng, (1, Hkv * G, D), act)
    al = (2.0 ** -np.arange(4, 4 + Hkv * G)).astype(np.float32) if slopes else None
    L = cuda(np.array([n], np.int32))
    kw = dict(first=1, last=2, alibi_slopes=cuda(al))
    got, other = fb.page_select(q, cache, bounds, L, 20, scale=-0.125, **kw), fb.page_select(-q, cache, bounds, L, 20, scale=0.125, **kw)
    assert torch.equal(got, other)
    for h in range(Hkv):
        want = E.select(-qa[0, h * G:(h + 1) * G], codes[table[0], h], scales[table[0], h], n, n, 1, G, 20, 0.125, 1, 2,
                        None if al is None else al[h * G:(h + 1) * G])
        assert got[0, h].tolist() == want, h
    assert fb.fa_back_get_error() == 0


def test_the_page_that_takes_nearly_all_of_the_attention_is_chosen(fb):
    """One page holds the key -q, whose score is the largest with a negative scale: attention over the chosen pages is that over all."""
    p = R.Paged(1, (800,), 1, 64, 64, R.synth.TYPE_F32, R.synth.TYPE_F32, 8, k_amp=0.1)
    q, qa = act_array(np.random.default_rng(1), (1, 1, 64), "f32")
    p.kd[0][333, 0] = -qa[0, 0].astype(np.float64)
    p.k[p.table[0, 333 // 8], 333 % 8, 0] = np.frombuffer((-qa[0, 0]).tobytes(), np.uint8)
    cache, L = p.on_gpu(fb, torch), cuda(np.array([800], np.int32))
    bounds = fb.PageBounds.of(cache)
    fb.page_bounds(cache, bounds, L)
    pages = fb.page_select(q, cache, bounds, L, 1, scale=-1.0, first=0, last=0)
    assert pages.tolist() == [[[333 // 8]]]
    x = -(p.kd[0][:, 0] @ qa[0, 0].astype(np.float64))
    assert np.exp(np.delete(x, 333) - x[333]).sum() < 1e-9  # what the other keys weigh
    O, _, mag, smag = R.decode(p, qa, -1.0)
    tol, _ = R.decode_tolerance(p, mag, smag, "f32")
    for which in (pages, None):
        got = fb.paged_decode(q, cache, L, scale=-1.0, pages=which)["O"].cpu().numpy()
        assert (np.abs(got - O) <= tol + 1e-9 * np.abs(p.vd[0]).max()).all()
