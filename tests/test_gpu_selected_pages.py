"""Attention over selected pages on the GPU: every kernel of it against 64-bit numpy, with the workspace that callers are told to
bring.  Tolerances are those of the single-token attention, and a rounding of the output's type."""
import numpy as np
import pytest

import paged_ref as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_paged_ext import act_array, cuda, fb, half_step, over_pages, within  # noqa: E402,F401

TYPES = ("f32", "f16", "q8_0", "q4_0")


def some_pages(rng, lens, Hkv, page, K):
    """[B][Hkv][K]: different pages of the sequence in any order, the last one often among them, some places empty."""
    pages = np.full((len(lens), Hkv, K), -1, np.int32)
    for b, L in enumerate(lens):
        n = -(-max(L, 0) // page)
        for hk in range(Hkv):
            m = min(K, n)
            mine = rng.permutation(n)[:m].astype(np.int32)
            if m and n - 1 not in mine:
                mine[rng.integers(0, m)] = n - 1
            mine[rng.random(m) < 0.1] = -1
            pages[b, hk, :m] = mine
    return pages


def check(fb, p, H, pages, act, softcap=0.0, al=None, sk=None, seed=0, workspace=None):
    rng = np.random.default_rng(seed)
    cache, n = p.on_gpu(fb, torch), cuda(np.array(p.lens, np.int32))
    q, qa = act_array(rng, (len(p.lens), H, p.D), act)
    scale = p.D ** -0.5
    got = fb.paged_decode(q, cache, n, scale=scale, softcap=softcap, alibi_slopes=cuda(al), sinks=cuda(sk), pages=cuda(pages), workspace=workspace)
    live = [b for b, L in enumerate(p.lens) if L >= 0]
    O, lse, mag, smag = over_pages(p, {(b, hk): pages[b, hk] for b in range(len(p.lens)) for hk in range(p.Hkv)}, qa, scale, softcap, al, sk)
    tol_O, tol_lse = R.decode_tolerance(p, mag, smag, act)
    within(got["O"].float().cpu().numpy()[live], O[live], tol_O[live] + half_step(act, O[live]), "O")
    within(got["lse"].cpu().numpy()[live], lse[live], tol_lse[live], "lse")
    assert fb.fa_back_get_error() == 0
    return cache, q, n, got


@pytest.mark.parametrize("B, Hkv, H, page, K, L", [(48, 1, 1, 16, 64, 8000), (8, 8, 8, 64, 64, 6000)])
def test_the_types_whose_kernels_run_more_ctas_than_the_plain_ones(fb, B, Hkv, H, page, K, L):
    """Keys of 64 components in q8_0 and values of 256 in f32 take three CTAs an SM over selected pages, two over all: more partial
    sums.  The size that fa_paged_decode_workspace_size() gives does for both."""
    rng = np.random.default_rng(B)
    lens = [int(x) for x in rng.integers(L // 2, L, B)]
    p = R.Paged(B, lens, Hkv, 64, 256, R.synth.TYPE_Q8_0, R.synth.TYPE_F32, page)
    pages = some_pages(rng, lens, Hkv, page, K)
    cache, q, n, got = check(fb, p, H, pages, "f32")
    again = fb.paged_decode(q, cache, n, scale=64 ** -0.5, pages=cuda(pages), workspace=fb.Workspace())
    assert torch.equal(got["O"], again["O"]) and torch.equal(got["lse"], again["lse"])


@pytest.mark.parametrize("page, K, lens", [(40, 64, (100, 700, 39)), (5, 21, (9, 90)), (12, 7, (3, 300)), (1, 40, (70, 20))])
def test_distances_where_selected_keys_end_inside_a_tile(fb, page, K, lens):
    """ALiBi over lists longer than the sequence has pages: what stands behind them does not matter, nor do entries that are
    no page."""
    rng = np.random.default_rng(page)
    p = R.Paged(page, lens, 2, 64, 64, R.synth.TYPE_F16, R.synth.TYPE_F16, page)
    pages = some_pages(rng, lens, 2, page, K)
    al = (2.0 ** -np.arange(2, 6)).astype(np.float32)
    cache, q, n, got = check(fb, p, 4, pages, "f32", al=al)
    for b, L in enumerate(lens):
        m = -(-L // page)
        pages[b, :, m:] = rng.integers(-2 ** 31, 2 ** 31, pages[b, :, m:].shape)  # behind the sequence's pages
        pages[b, :, :m][pages[b, :, :m] < 0] = 2 ** 31 - 1
    again = fb.paged_decode(q, cache, n, scale=64 ** -0.5, alibi_slopes=cuda(al), pages=cuda(pages))
    assert torch.equal(got["O"], again["O"]) and torch.equal(got["lse"], again["lse"])
    assert fb.fa_back_get_error() == 0


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Dv", [64, 128, 256])
def test_every_pair_of_types(fb, D, Dv):
    """Each kernel over selected pages: seeded lengths, page sizes (boxes of 16 and 8 rows, single rows), lists and extensions."""
    r = np.random.default_rng(D + 3 * Dv)
    pick = lambda *a: a[int(r.integers(len(a)))]  # noqa: E731
    for kt in range(4):
        for vt in range(4):
            Hkv, G, K, act = pick(1, 2, 3), pick(1, 3, 8, 9), pick(1, 5, 20, 60), pick("f32", "f16", "bf16")
            page = pick(8, 16, 24, 64, 5, 12)
            if page * Hkv * R.synth.row_bytes(kt, D) % 16 or page * Hkv * R.synth.row_bytes(vt, Dv) % 16:
                page = 16
            lens = [int(x) for x in np.exp(r.uniform(-0.5, np.log(3000), int(r.integers(1, 6))))] + [0]
            p = R.Paged(16 * D + 4 * kt + vt, lens, Hkv, D, Dv, kt, vt, page)
            H = G * Hkv
            al = (2.0 ** -np.linspace(2, 9, H)).astype(np.float32) if pick(True, False) else None
            sk = r.standard_normal(H).astype(np.float32) if pick(True, False) else None
            check(fb, p, H, some_pages(r, lens, Hkv, page, K), act, pick(0.0, 0.0, 20.0), al, sk, seed=kt)
