"""The operators around the paged cache on the GPU: keys stored through either path, positions of several axes,
page lists, page bounds, page selection and attention over selected pages, against 64-bit numpy.

Tolerances are bounds from the roundings that each operator makes, written beside them; whole numbers are equal.
"""
import numpy as np
import pytest

import paged_ext_ref as E
import paged_ref as R
import synth

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
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


# ------------------------------------------------------------------------------------------------
# positions of several axes

def half_step(act, ref):
    return 0.0 if act == "f32" else torch.finfo(DT[act]).eps / 2 * np.abs(ref) * 1.01 + torch.finfo(DT[act]).smallest_normal * 2.0 ** -8


def act_array(rng, shape, act):
    t = torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(DT[act]).cuda()
    return t, t.float().cpu().numpy()


def within(got, ref, tol, what=""):
    got = np.asarray(got, np.float64)
    fin = np.isfinite(ref)
    assert np.array_equal(np.isneginf(got), np.isneginf(ref)), what
    off, tol = np.abs(got[fin] - ref[fin]), np.broadcast_to(tol, ref.shape)[fin]
    bad = ~(off <= tol)
    assert not bad.any(), (what, int(bad.sum()), off[bad][:4], tol[bad][:4])


AXES = {  # N, H, Hkv, D, act, out, sections, interleaved, halves, weights, fused
    "one_token": (1, 1, 1, 64, "f32", "f32", (16, 8, 8), False, True, True, False),
    "odd": (37, 6, 2, 128, "f32", "f32", (16, 24, 24), False, True, True, False),
    "in_turn": (33, 5, 5, 256, "bf16", "bf16", (44, 42, 42), True, True, True, True),
    "pairs": (50, 3, 1, 64, "f32", "bf16", (9, 23), False, False, True, False),
    "partial_pairs": (33, 4, 3, 128, "bf16", "f16", (5, 1, 0, 11), True, False, True, True),
    "partial_halves": (33, 4, 1, 256, "f16", "f32", (8, 8, 4, 12), False, True, True, True),
    "no_norm": (21, 4, 2, 128, "f32", "f32", (32, 32), True, True, False, False),
    "eight_axes": (700, 9, 3, 64, "bf16", "f32", (4,) * 8, True, True, True, True),
    "queries_only": (40, 7, 0, 256, "f32", "f32", (60, 4), False, False, True, False),
}


def axes_inputs(fb, name):
    N, H, Hkv, D, act, out, sections, turn, halves, weights, fused = AXES[name]
    rng = np.random.default_rng(sorted(AXES).index(name) + 300)
    if fused:
        x, xa = act_array(rng, (N, H + 2 * Hkv + 1, D), act)
        q, k, qa, ka = x[:, :H], x[:, H:H + Hkv], xa[:, :H], xa[:, H:H + Hkv]
    else:
        (q, qa), (k, ka) = act_array(rng, (N, H, D), act), act_array(rng, (N, Hkv, D), act)
    A = len(sections)
    pos = rng.integers(-5, 2000000, (A, N)).astype(np.int32)
    wide = torch.full((A, N + 3), 77, dtype=torch.int32, device="cuda")  # the axes' rows lie apart
    wide[:, 1:N + 1] = cuda(pos)
    w = [(1.0 + 0.2 * rng.standard_normal(D)).astype(np.float32) if weights else None for _ in range(2)]
    axes = fb.rope_sections(sections, interleaved=turn)
    kw = dict(wq=cuda(w[0]), wk=cuda(w[1]) if Hkv else None, eps=1e-6, rope=fb.rope_frequencies(2 * sum(sections)),
              rope_style=int(halves), rope_axes=axes)
    return (N, H, Hkv, D, act, out, halves), q, k if Hkv else None, qa, ka, pos, wide[:, 1:N + 1], w, axes.cpu().numpy(), kw, rng


@pytest.mark.parametrize("name", sorted(AXES))
def test_norm_rope_axes(fb, name):
    (N, H, Hkv, D, act, out, halves), q, k, qa, ka, pos, p, w, axes, kw, _ = axes_inputs(fb, name)
    got = fb.qk_norm_rope(q, k, p, dtype=DT[out], **kw)
    n_rot = 2 * len(axes)
    for n, x, wt in (("q", qa, w[0]), ("k", ka, w[1])):
        if not x.shape[1]:
            assert got[n] is None
            continue
        y = R.norm(x, wt, 1e-6) if wt is not None else x.astype(np.float64)
        ref = E.rotate_axes(y, pos, axes, 10000.0, halves)
        # r: sum of squares in chains of 8 and 5 (13 u, halved), its root 2 u, two products; cos and sin within 3 u
        # and the 32-bit angle (2 u): under 20 u of the pair's magnitude
        mag = np.abs(y)
        i = np.arange(n_rot // 2)
        f, s = (i, i + n_rot // 2) if halves else (2 * i, 2 * i + 1)
        mag[..., f] = mag[..., s] = mag[..., f] + mag[..., s]
        within(got[n].float().cpu().numpy(), ref, 20 * U * mag + half_step(out, ref), n)
    assert fb.fa_back_get_error() == 0


def back_reference(x, w, gy, pos, axes, halves, eps=1e-6):
    x, gy = x.astype(np.float64), gy.astype(np.float64)
    g = E.rotate_axes(gy, pos, axes, 10000.0, halves, -1.0)
    if w is None:
        return g, None, None, g
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    h = g * w.astype(np.float64)
    return r * (h - x * r * r * (h * x).mean(-1, keepdims=True)), (g * x * r).sum((0, 1)), r, g


@pytest.mark.parametrize("name", sorted(AXES))
def test_norm_rope_axes_backward(fb, name):
    (N, H, Hkv, D, act, out, halves), q, k, qa, ka, pos, p, w, axes, kw, rng = axes_inputs(fb, name)
    (gq, gqa), (gk, gka) = act_array(rng, (N, H, D), out), act_array(rng, (N, Hkv, D), out)
    got = fb.qk_norm_rope_backward(gq, gk if Hkv else None, q, k, p, **kw)
    for n, x, wt, gy in (("q", qa, w[0], gqa), ("k", ka, w[1], gka)):
        if not x.shape[1]:
            assert "d" + n not in got
            continue
        dx, dw, r, g = back_reference(x, wt, gy, pos, axes, halves)
        gmax = np.abs(g).max(-1, keepdims=True) + np.abs(gy).max(-1, keepdims=True)
        if wt is None:
            within(got["d" + n].float().cpu().numpy(), dx, 20 * U * gmax + half_step(act, dx), "d" + n)
            continue
        # as the forward's, twice (g, then the product with r), and the mean of h o x: 20 u of its magnitudes
        x64, wm = x.astype(np.float64), np.abs(wt).max()
        mag = r * (gmax * wm + np.abs(x64) * r * r * (gmax * wm * np.abs(x64)).mean(-1, keepdims=True))
        within(got["d" + n].float().cpu().numpy(), dx, 48 * U * mag + half_step(act, dx), "d" + n)
        # dw: terms within 40 u of theirs, summed in chains of at most rows / 8 + 400 additions
        terms = (gmax * np.abs(x64) * r).sum((0, 1))
        within(got["dw" + n].cpu().numpy(), dw, (40 + N * x.shape[1] / 8 + 400) * U * terms, "dw" + n)
    assert fb.fa_back_get_error() == 0


def test_norm_rope_axes_backward_against_differences(fb):
    """<dx, v> + <dw, u> is the central difference of <gy, y> along (v, u), taken in 64 bits."""
    (N, H, Hkv, D, act, out, halves), q, k, qa, ka, pos, p, w, axes, kw, rng = axes_inputs(fb, "odd")
    (gq, gqa), (gk, gka) = act_array(rng, (N, H, D), "f32"), act_array(rng, (N, Hkv, D), "f32")
    got = fb.qk_norm_rope_backward(gq, gk, q, k, p, **kw)
    for n, x, wt, gy in (("q", qa, w[0], gqa), ("k", ka, w[1], gka)):
        v, uw, e = rng.standard_normal(x.shape), rng.standard_normal(D), 1e-5
        x, wt, gy = (a.astype(np.float64) for a in (x, wt, gy))
        f = lambda t: (gy * E.rotate_axes(R.norm(x + t * v, wt + t * uw, 1e-6), pos, axes, 10000.0, halves)).sum()  # noqa: E731
        want = (f(e) - f(-e)) / (2 * e)
        dx, dw = got["d" + n].double().cpu().numpy(), got["dw" + n].double().cpu().numpy()
        have = (dx * v).sum() + (dw * uw).sum()
        # dx within 48 u of magnitudes of a few, over N heads D terms of mixed signs; the difference itself is e^2
        assert abs(have - want) <= 1e-4 * np.sqrt(x.size) + 1e-6 * abs(want)


@pytest.mark.parametrize("D, halves", [(64, True), (128, False), (256, True)])
def test_one_position_for_all_axes_is_the_plain_rotation(fb, D, halves):
    """Bit for bit, forward, backward and append; and each axis alone, with an axis number beyond the last one."""
    rng = np.random.default_rng(D)
    N, H, Hkv = 45, 4, 2
    (q, _), (k, _), (v, _) = (act_array(rng, (N, h, D), "bf16") for h in (H, Hkv, Hkv))
    w = cuda((1.0 + 0.2 * rng.standard_normal(D)).astype(np.float32))
    pos = cuda(rng.permutation(4 * N)[:N].astype(np.int32))
    seq = torch.zeros(N, dtype=torch.int32, device="cuda")
    kw = dict(rope=fb.rope_frequencies(D), rope_style=int(halves))
    one = fb.qk_norm_rope(q, k, pos, wq=w, wk=w, **kw)
    back = fb.qk_norm_rope_backward(one["q"], one["k"], q, k, pos, wq=w, wk=w, **kw)
    a = empty_cache(fb, 1, 12, 16, Hkv, D, D, fb.FA_Q8_0, fb.FA_F16)
    fb.cache_append(k, v, a, seq, pos, k_norm=w, **kw)
    for axes, p in ((fb.rope_sections([D // 8, D // 8, D // 4]), pos.expand(3, N)),
                    (torch.full((D // 2,), 9, dtype=torch.uint8, device="cuda"), torch.stack([pos * 0 - 3, pos]))):
        several = fb.qk_norm_rope(q, k, p, wq=w, wk=w, rope_axes=axes, **kw)
        back2 = fb.qk_norm_rope_backward(one["q"], one["k"], q, k, p, wq=w, wk=w, rope_axes=axes, **kw)
        b = empty_cache(fb, 1, 12, 16, Hkv, D, D, fb.FA_Q8_0, fb.FA_F16)
        fb.cache_append(k, v, b, seq, pos, k_norm=w, rope_axes=axes, rope_pos=p, **kw)
        assert all(torch.equal(one[n], several[n]) for n in one) and all(torch.equal(back[n], back2[n]) for n in back)
        assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v)


@pytest.mark.parametrize("D, halves, sections, kt, act", [(64, True, (16, 8, 8), "f32", "f32"), (128, False, (3, 20), "q8_0", "bf16"),
                                                         (256, True, (24, 20, 20), "q4_0", "f16")])
def test_append_axes(fb, D, halves, sections, kt, act):
    """Rotated by one set of positions, stored at another: what the rotation and a plain append store."""
    rng = np.random.default_rng(D + 1)
    T, Hkv, t = 83, 3, {"f32": fb.FA_F32, "q8_0": fb.FA_Q8_0, "q4_0": fb.FA_Q4_0}[kt]
    (k, _), (v, _) = (act_array(rng, (T, Hkv, D), act) for _ in range(2))
    w = cuda((1.0 + 0.2 * rng.standard_normal(D)).astype(np.float32))
    at = rng.permutation(2 * 6 * 16)[:T].astype(np.int32)
    seq, pos = cuda(at % 2), cuda(at // 2)
    seq[5], pos[9] = -1, -7  # padding
    p = cuda(rng.integers(0, 100000, (len(sections), T)).astype(np.int32))
    kw = dict(rope=fb.rope_frequencies(2 * sum(sections)), rope_style=int(halves), rope_axes=fb.rope_sections(sections, interleaved=True))
    y = fb.qk_norm_rope(k, None, p, wq=w, dtype=torch.float32, **kw)["q"]
    one, two = (empty_cache(fb, 2, 6, 16, Hkv, D, D, t, fb.FA_F32) for _ in range(2))
    fb.cache_append(k, v, one, seq, pos, k_norm=w, rope_pos=p, **kw)
    fb.cache_append(y, v.float(), two, seq, pos)
    assert torch.equal(one.k, two.k) and torch.equal(one.v, two.v) and bool(one.k.any())
    assert fb.fa_back_get_error() == 0


# ------------------------------------------------------------------------------------------------
# page lists

def lists_of(fb, rng, B, width, num_pages, page, fill, empty=0.1):
    """Random requests that hold about a share `fill` of the pages; the tensors and the same as lists."""
    order = rng.permutation(num_pages).tolist()
    table, lens = np.full((B, width), -1, np.int32), np.zeros(B, np.int64)
    left = int(fill * num_pages)
    for b in range(B):
        n = int(rng.integers(0, width * page + 1))
        pages = -(-n // page)
        if rng.random() < empty:
            lens[b] = -1
        elif pages <= left:
            left -= pages
            lens[b] = n
            table[b, :pages] = [order.pop() for _ in range(pages)]
    free = np.full(num_pages, -1, np.int32)
    free[:len(order)] = order
    t = [cuda(x.astype(np.int32)) for x in (table, lens, free, np.array([len(order)]))]
    return fb.PageLists(*t, page_size=page), E.Lists(table, lens.tolist(), order, num_pages, page)


def same_lists(lists, ref):
    n = int(lists.num_free)
    assert lists.page_table.tolist() == ref.table and lists.seq_lens.tolist() == ref.lens
    assert n == len(ref.stack) and lists.free[:n].tolist() == ref.stack


@pytest.mark.parametrize("B, width, page, tokens, num_pages", [
    (1, 1, 1, 1, 1), (1, 5, 16, 40, 9), (7, 9, 5, 30, 40), (64, 40, 16, 3, 900), (100, 3, 64, 200, 200), (1023, 4, 7, 9, 2500),
    (1024, 4, 7, 9, 3000), (1025, 4, 7, 9, 3000), (2600, 6, 3, 20, 9000), (9, 3000, 16, 30000, 20000)])
def test_pages_extend_and_trim(fb, B, width, page, tokens, num_pages):
    """Steps of random requests: some find no pages, some no room in their row, some end behind T; then trims, some to
    nothing, some that leave a request as it is."""
    rng = np.random.default_rng(B + width)
    lists, ref = lists_of(fb, rng, B, width, num_pages, page, 0.4)
    for step in range(5):
        news = np.where(rng.random(B) < 0.2, rng.integers(-2, 1, B), rng.integers(1, tokens + 1, B)).astype(np.int32)
        need = int(np.maximum(news, 0)[np.array(ref.lens) >= 0].sum())
        T = [need, need + 5, need // 2, need, 0][step]
        got = fb.pages_extend(lists, cuda(news), T)
        want = ref.extend(news.tolist(), T)
        for n, x in want.items():
            assert got[n].tolist() == x, (step, n)
        same_lists(lists, ref)
        lens = np.array(ref.lens)
        keep = np.where(rng.random(B) < 0.3, -1, np.where(rng.random(B) < 0.3, 0, lens - rng.integers(-3, tokens + 2, B))).astype(np.int32)
        keep = np.where((keep < 0) & (rng.random(B) < 0.5), 0, keep).astype(np.int32)
        fb.pages_trim(lists, cuda(keep))
        ref.trim(keep.tolist())
        same_lists(lists, ref)
    assert fb.fa_back_get_error() == 0


def test_page_lists_without_requests_or_pages(fb):
    none = fb.PageLists.empty(0, 3, 5, 16)
    got = fb.pages_extend(none, torch.empty(0, dtype=torch.int32, device="cuda"), 7)
    assert got["starts"].tolist() == [0] and got["seq"].tolist() == [-1] * 7 and got["first"].numel() == 0
    fb.pages_trim(none, torch.empty(0, dtype=torch.int32, device="cuda"))
    assert none.num_free.tolist() == [5]
    for lists in (fb.PageLists.empty(2, 0, 5, 16), fb.PageLists.empty(2, 3, 0, 16)):
        lists.seq_lens.zero_()
        got = fb.pages_extend(lists, torch.full((2,), 9, dtype=torch.int32, device="cuda"), 10000)
        assert got["starts"].tolist() == [0, 9, 18] and got["first"].tolist() == [-1, -1] and got["row"].tolist() == [-1] * 10000
        assert lists.seq_lens.tolist() == [0, 0]
    assert fb.fa_back_get_error() == 0


def test_sums_of_tokens_beyond_32_bits(fb):
    """Requests for more tokens than an int holds: refused, and those before and behind them that fit T are not disturbed."""
    lists = fb.PageLists.empty(5, 4, 20, 16)
    lists.seq_lens.copy_(torch.tensor([0, 0, 0, 5, 0]))
    lists.page_table[3, 0] = 19
    news = torch.tensor([20, 0, 2 ** 31 - 1, 2 ** 31 - 1, 2], dtype=torch.int32, device="cuda")
    got = fb.pages_extend(lists, news, 30)
    assert got["starts"].tolist() == [0, 20, 20, 30, 30, 30] and got["first"].tolist() == [0, -1, -1, -1, -1]
    assert got["seq"].tolist() == [0] * 20 + [-1] * 10 and lists.seq_lens.tolist() == [20, 0, 0, 5, 0] and lists.num_free.tolist() == [18]


def test_trim_undoes_extend_and_requests_come_and_go(fb):
    lists = fb.PageLists.empty(4, 8, 20, 16)
    assert lists.free[:3].tolist() == [19, 18, 17] and lists.num_free.tolist() == [20]
    lists.seq_lens.copy_(torch.tensor([0, -1, 0, 0]))
    got = fb.pages_extend(lists, cuda(np.array([20, 5, 1, 0], np.int32)), 21)
    assert lists.seq_lens.tolist() == [20, -1, 1, 0] and lists.page_table[0, :3].tolist() == [0, 1, -1]
    assert got["first"].tolist() == [0, -1, 0, -1] and got["starts"].tolist() == [0, 20, 20, 21, 21]
    before = [t.clone() for t in (lists.page_table, lists.seq_lens, lists.free, lists.num_free)]
    keep = lists.seq_lens.clone()
    fb.pages_extend(lists, cuda(np.array([100, 9, 40, 7], np.int32)), 147)
    assert lists.num_free.tolist() == [20 - 8 - 3 - 1]
    fb.pages_trim(lists, keep)
    assert all(torch.equal(a, b) for a, b in zip(before, (lists.page_table, lists.seq_lens, lists.free, lists.num_free)))
    fb.pages_trim(lists, torch.zeros_like(keep))
    assert lists.num_free.tolist() == [20] and sorted(lists.free.tolist()) == list(range(20))
    assert lists.seq_lens.tolist() == [0, -1, 0, 0] and bool((lists.page_table == -1).all())


def test_page_lists_that_are_wrong_are_reported_and_stay_in_bounds(fb):
    """A page given back twice, a count outside the pool, page numbers that are none."""
    def lists(table, lens, free, n):
        return fb.PageLists(*(cuda(np.array(x, np.int32)) for x in (table, lens, free, [n])), page_size=4)
    one = lists([[0, 1], [0, 1]], [8, 8], [2, -1, -1], 1)  # three pages, four given back
    fb.pages_trim(one, cuda(np.array([0, 0], np.int32)))
    assert fb.STATUS[fb.fa_back_get_error()] == "FA_ERR_PAGE" and one.num_free.tolist() == [3] and fb.fa_back_get_error() == 0
    two = lists([[-1, -1]], [0], [2, 1, 0], 99)
    got = fb.pages_extend(two, cuda(np.array([8], np.int32)), 8)
    assert two.num_free.tolist() == [1] and two.page_table.tolist() == [[0, 1]] and got["row"].tolist() == list(range(8))
    three = lists([[-1, -1]], [0], [2, 1, 0], -5)
    got = fb.pages_extend(three, cuda(np.array([8], np.int32)), 8)
    assert three.num_free.tolist() == [0] and got["first"].tolist() == [-1] and got["seq"].tolist() == [-1] * 8
    assert fb.fa_back_get_error() == 0
    four = lists([[7, -1]], [2], [1, 1, -3], 3)  # the request's first page is none, and so is the next one to be taken
    got = fb.pages_extend(four, cuda(np.array([4], np.int32)), 4)
    assert got["row"].tolist() == [-1] * 4 and got["pos"].tolist() == [2, 3, 4, 5] and four.page_table.tolist() == [[7, -3]]
    assert fb.STATUS[fb.fa_back_get_error()] == "FA_ERR_PAGE"


# ------------------------------------------------------------------------------------------------
# bounds

TYPES = {"f32": 0, "f16": 1, "q8_0": 2, "q4_0": 3}


def want_bounds(p, b, j):
    """Codes and scales [Hkv] of page j of sequence b of a paged_ref cache."""
    rows = p.kd[b][j * p.page:(j + 1) * p.page]
    got = [E.bounds(rows[:, h]) for h in range(p.Hkv)]
    return np.stack([c for c, _ in got]), np.stack([s for _, s in got])


@pytest.mark.parametrize("kt", sorted(TYPES))
@pytest.mark.parametrize("D, Hkv, page, lens", [(64, 1, 16, (37, 0, 1, 16, -1, 200)), (128, 3, 40, (41, 40, 39)), (256, 2, 8, (100, 7)),
                                                (64, 2, 64, (1000,)), (128, 5, 2, (5, 0))])
def test_page_bounds(fb, kt, D, Hkv, page, lens):
    """All pages; rows behind the lengths, and pages of nobody, are NaN.  Then only pages from a position on."""
    p = R.Paged(D + page, lens, Hkv, D, 64, TYPES[kt], TYPES["f16"], page if TYPES[kt] != 3 else max(page, 8), k_amp=3.0)
    cache = p.on_gpu(fb, torch)
    bounds = fb.PageBounds.of(cache)
    bounds.codes.fill_(99), bounds.scales.fill_(-1)
    n = cuda(np.array(lens, np.int32))
    fb.page_bounds(cache, bounds, n)
    codes, scales = bounds.codes.cpu().numpy(), bounds.scales.cpu().numpy()
    held = np.zeros(len(codes), bool)
    for b, L in enumerate(lens):
        for j in range(-(-max(L, 0) // p.page)):
            at = p.table[b, j]
            held[at] = True
            c, s = want_bounds(p, b, j)
            assert np.array_equal(codes[at], c) and np.array_equal(scales[at], s), (b, j)
            vals = codes[at].astype(np.float64) * s.repeat(32, -1)[:, None].astype(np.float64)
            rows = p.kd[b][j * p.page:(j + 1) * p.page]
            # they bound the keys: but for the roundings of hi / d and of d, 3 u of the block's largest (127 d)
            slack = 127 * s.repeat(32, -1) * 3 * U
            assert (vals[:, 0] >= rows.max(0) - slack).all() and (vals[:, 1] <= rows.min(0) + slack).all()
    assert (codes[~held] == 99).all() and (scales[~held] == -1).all()
    bounds.codes.fill_(99)
    first = np.array([max(L - 1 - i, -1) for i, L in enumerate(lens)], np.int32)
    fb.page_bounds(cache, bounds, n, first=cuda(first))
    again = bounds.codes.cpu().numpy()
    for b, L in enumerate(lens):
        for j in range(-(-max(L, 0) // p.page)):
            done = 0 <= first[b] < L and j >= first[b] // p.page
            assert np.array_equal(again[p.table[b, j]], codes[p.table[b, j]]) if done else (again[p.table[b, j]] == 99).all(), (b, j)
    assert fb.fa_back_get_error() == 0


def test_page_bounds_of_values_that_are_not_finite_or_tiny(fb):
    k = torch.zeros(3, 4, 1, 64, device="cuda")
    k[0, 1, 0, 3], k[0, 2, 0, 40] = float("nan"), float("inf")  # one block with a NaN, one with an infinity
    k[0, :, 0, 5] = torch.tensor([1.0, -2.0, 0.5, 0.0], device="cuda")
    k[1] = 1e-31
    k[2, :, 0, 33] = float("nan")  # nothing but NaN in a component
    raw = k.view(torch.uint8).view(3, 4, 1, 256)
    cache = fb.PagedCache(raw, fb.FA_F32, raw.clone(), fb.FA_F32, cuda(np.array([[0, 1, 2]], np.int32)), D=64, Dv=64)
    bounds = fb.PageBounds.of(cache)
    fb.page_bounds(cache, bounds, cuda(np.array([12], np.int32)))
    c, s = bounds.codes.cpu(), bounds.scales.cpu()
    assert c[0, 0, 0, :32].tolist() == [0] * 5 + [64] + [0] * 26 and c[0, 0, 1, :32].tolist() == [0] * 5 + [-127] + [0] * 26
    assert s[0, 0, 0].item() == np.float32(2) / np.float32(127) and s[0, 0, 1].item() == float("inf")
    assert (c[0, 0, 0, 32:] == 127).all() and (c[0, 0, 1, 32:] == -127).all()
    assert not c[1].any() and not s[1].any() and s[2, 0].tolist() == [0.0, float("inf")]
    bad = fb.PagedCache(raw, fb.FA_F32, raw.clone(), fb.FA_F32, cuda(np.array([[0, 3, -1]], np.int32)), D=64, Dv=64)
    fb.page_bounds(bad, bounds, cuda(np.array([99], np.int32)))  # invalid pages, a length beyond the table
    assert fb.STATUS[fb.fa_back_get_error()] == "FA_ERR_PAGE"


# ------------------------------------------------------------------------------------------------
# selection

def check_select(p, codes, scales, q, pages, lens, H, K, scale, first, last, slopes=None):
    G = H // p.Hkv
    for b, L in enumerate(lens):
        if L < 0:
            assert (pages[b] == -77).all()
            continue
        n = -(-L // p.page)
        at = p.table[b, :n]
        for h in range(p.Hkv):
            want = E.select(q[b, h * G:(h + 1) * G], codes[at, h], scales[at, h], n, L, p.page, G, K, scale, first, last,
                            None if slopes is None else slopes[h * G:(h + 1) * G])
            assert pages[b, h].tolist() == want + [-1] * (K - len(want)), (b, h)


@pytest.mark.parametrize("D, Hkv, H, page, lens, K, first, last, act, alibi", [
    (64, 1, 1, 16, (700, 0, 1, 16, -1, 321), 5, 1, 1, "f32", False), (128, 2, 8, 8, (400, 399, 7), 7, 0, 0, "bf16", True),
    (256, 3, 3, 8, (130, 300), 1, 0, 1, "f16", False), (128, 1, 40, 16, (900,), 9, 3, 6, "f32", True), (64, 2, 2, 2, (3000, 50), 33, 1, 2, "bf16", False),
    (256, 1, 17, 40, (2000, 1999), 16, 2, 0, "f32", False)])
def test_page_select(fb, D, Hkv, H, page, lens, K, first, last, act, alibi):
    """Equal to the definition's choice, every page of it; the queries are a view."""
    p = R.Paged(D + K, lens, Hkv, D, 64, 1, 1, page, k_amp=2.0)
    cache = p.on_gpu(fb, torch)
    bounds = fb.PageBounds.of(cache)
    n = cuda(np.array(lens, np.int32))
    fb.page_bounds(cache, bounds, n)
    rng = np.random.default_rng(K)
    x, xa = act_array(rng, (len(lens), H + 3, D), act)
    slopes = (2.0 ** -np.arange(1, H + 1)).astype(np.float32) if alibi else None
    out = torch.full((len(lens), Hkv, K), -77, dtype=torch.int32, device="cuda")
    got = fb.page_select(x[:, 2:H + 2], cache, bounds, n, K, scale=0.3, first=first, last=last, alibi_slopes=cuda(slopes), out=out)
    assert got is out
    check_select(p, bounds.codes.cpu().numpy(), bounds.scales.cpu().numpy(), xa[:, 2:H + 2], got.cpu().numpy(), lens, H, K, 0.3, first, last, slopes)
    assert fb.fa_back_get_error() == 0


def bounded_cache(fb, rng, n, D=64, Hkv=1, page=1, codes=None):
    """A cache of one sequence with n pages and given or random bounds; no keys to speak of."""
    raw = torch.zeros(n, page, Hkv, 2 * D, dtype=torch.uint8, device="cuda")
    table = rng.permutation(n).astype(np.int32)[None]
    cache = fb.PagedCache(raw, fb.FA_F16, raw, fb.FA_F16, cuda(table), D=D, Dv=D)
    codes = rng.integers(-127, 128, (n, Hkv, 2, D)).astype(np.int8) if codes is None else codes
    scales = rng.random((n, Hkv, D // 32)).astype(np.float32)
    return cache, fb.PageBounds(cuda(codes), cuda(scales)), codes, scales, table


@pytest.mark.parametrize("n, K, first, last", [(512, 511, 0, 0), (513, 64, 1, 2), (8192, 100, 0, 1), (8193, 100, 5, 0), (20000, 8192, 1, 1), (70001, 3, 1, 2)])
def test_page_select_of_many_pages(fb, n, K, first, last):
    """The keys in registers, and beyond; forced pages alone in the last case."""
    rng = np.random.default_rng(n)
    cache, bounds, codes, scales, table = bounded_cache(fb, rng, n)
    q, qa = act_array(rng, (1, 3, 64), "f32")
    got = fb.page_select(q, cache, bounds, cuda(np.array([n], np.int32)), K, scale=1.0, first=first, last=last)
    assert got[0, 0].tolist() == E.select(qa[0], codes[table[0], 0], scales[table[0], 0], n, n, 1, 3, K, 1.0, first, last)


@pytest.mark.parametrize("n, D, Hkv, G", [(1500, 128, 1, 8), (1500, 256, 2, 9), (40000, 64, 1, 20), (60000, 128, 2, 3), (60000, 256, 1, 17), (300, 256, 30, 2)])
def test_page_select_by_clusters_of_all_sizes_and_without(fb, n, D, Hkv, G):
    """Few sequences of many pages: clusters of eight CTAs, of twice the warps where SMs are free, and two launches where a
    sequence's keys do not fit shared memory; more than eight query heads add to what the first ones found."""
    rng = np.random.default_rng(n + D)
    cache, bounds, codes, scales, table = bounded_cache(fb, rng, n, D, Hkv, 1)
    q, qa = act_array(rng, (1, Hkv * G, D), "f16")
    got = fb.page_select(q, cache, bounds, cuda(np.array([n], np.int32)), 77, scale=0.1, first=2, last=3)
    for h in range(Hkv):
        assert got[0, h].tolist() == E.select(qa[0, h * G:(h + 1) * G], codes[table[0], h], scales[table[0], h], n, n, 1, G, 77, 0.1, 2, 3), h


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_are_exact_at_the_largest_codes(fb, D, sign):
    """All codes at the ends of their range, but for one that is one smaller from page to page: the sums of products differ by 127
    in half a million, and the order of the pages shows each."""
    rng = np.random.default_rng(D)
    n = 200
    codes = np.full((n, 1, 2, D), 127, np.int8)
    codes[:, :, 1] = -127
    down = rng.permutation(n)  # page i is down[i] below the largest
    for i in range(n):
        left = int(down[i])
        for j in range(0, 32):  # of the first block, at most 8 a component
            take = min(left, 8)
            codes[i, 0, 0 if sign > 0 else 1, j] -= sign * take
            left -= take
    cache, bounds, codes, scales, table = bounded_cache(fb, rng, n, D, 1, 1, codes=codes)
    bounds.scales.fill_(0.25), scales.fill(0.25)
    table = table[0]
    q = torch.full((1, 2, D), float(sign), device="cuda")
    got = fb.page_select(q, cache, bounds, cuda(np.array([n], np.int32)), 61, scale=1.0, first=0, last=0)
    assert got[0, 0].tolist() == sorted(i for i in range(n) if down[table[i]] < 61)


def test_page_select_of_queries_that_are_not_finite(fb):
    """Whatever is chosen is K different pages of the sequence."""
    rng = np.random.default_rng(9)
    cache, bounds, *_ = bounded_cache(fb, rng, 600)
    q, _ = act_array(rng, (1, 4, 64), "f32")
    for bad in (float("nan"), float("inf"), -3e38):
        for at in ((0, 0, 5), (0, slice(None), slice(None))):
            x = q.clone()
            x[at] = bad
            got = fb.page_select(x, cache, bounds, cuda(np.array([600], np.int32)), 50, scale=1.0)[0, 0].tolist()
            assert got == sorted(set(got)) and len(got) == 50 and got[0] == 0 and got[-1] == 599


def test_more_pages_asked_for_than_there_are(fb):
    p = R.Paged(12, (70, 3, 0), 2, 64, 64, 1, 1, 16)
    cache, n = p.on_gpu(fb, torch), cuda(np.array([70, 3, 0], np.int32))
    bounds = fb.PageBounds.of(cache)
    fb.page_bounds(cache, bounds, n)
    q, qa = act_array(np.random.default_rng(1), (3, 4, 64), "f32")
    pages = fb.page_select(q, cache, bounds, n, 1000, scale=1.0, first=500, last=500)
    assert all(pages[b, h].tolist() == list(range(m)) + [-1] * (1000 - m) for b, m in ((0, 5), (1, 1), (2, 0)) for h in range(2))
    got, want = fb.paged_decode(q, cache, n, scale=1.0, pages=pages), R.decode(p, qa, 1.0)
    tol_O, tol_lse = R.decode_tolerance(p, want[2], want[3], "f32")
    within(got["O"].cpu().numpy(), want[0], tol_O), within(got["lse"].cpu().numpy(), want[1], tol_lse)


def test_pools_beyond_32_bits(fb):
    """Page numbers whose rows and whose bounds lie more than 4 GB behind the pools' starts."""
    n, Hkv, D = (1 << 20) + 40, 8, 256
    k = torch.zeros(n, 1, Hkv, 2 * D, dtype=torch.uint8, device="cuda")
    table = torch.arange(n - 30, n, dtype=torch.int32, device="cuda")[None]
    rows = torch.randn(30, 1, Hkv, D, device="cuda").half()
    k[n - 30:] = rows.view(torch.uint8).view(30, 1, Hkv, 2 * D)
    cache = fb.PagedCache(k, fb.FA_F16, k, fb.FA_F16, table, D=D, Dv=D)
    bounds, L = fb.PageBounds.of(cache), cuda(np.array([30], np.int32))
    fb.page_bounds(cache, bounds, L)
    v = rows[:, 0].double().cpu().numpy()
    for i in (0, 29):
        for h in range(Hkv):
            c, s = E.bounds(v[i:i + 1, h])
            assert np.array_equal(bounds.codes[n - 30 + i, h].cpu().numpy(), c) and np.array_equal(bounds.scales[n - 30 + i, h].cpu().numpy(), s)
    assert not bounds.codes[:n - 30].any()
    q, qa = act_array(np.random.default_rng(2), (1, Hkv, D), "f32")
    pages = fb.page_select(q, cache, bounds, L, 7, scale=0.06)
    codes, scales = bounds.codes[n - 30:].cpu().numpy(), bounds.scales[n - 30:].cpu().numpy()
    for h in range(Hkv):
        assert pages[0, h].tolist() == E.select(qa[0, h:h + 1], codes[:, h], scales[:, h], 30, 30, 1, 1, 7, 0.06, 1, 1)
    got = fb.paged_decode(q, cache, L, scale=0.06, pages=pages)["O"][0].double().cpu().numpy()
    for h in range(Hkv):
        r = v[pages[0, h].cpu().numpy(), h]
        w = np.exp(0.06 * (r @ qa[0, h].astype(np.float64)))
        assert np.abs(got[h] - w @ r / w.sum()).max() < 1e-4
    assert fb.fa_back_get_error() == 0


@pytest.mark.parametrize("n, K", [(700, 50), (9000, 300)])
def test_page_select_takes_the_lowest_of_equal_pages(fb, n, K):
    """Scores of few different values, of one, and of none (a query of zeros: all scores are 0, of either sign)."""
    rng = np.random.default_rng(n)
    kinds = rng.integers(-3, 4, (5, 1, 2, 64)).astype(np.int8)
    cache, bounds, codes, scales, table = bounded_cache(fb, rng, n, codes=kinds[rng.integers(0, 5, n)])
    bounds.scales.fill_(0.5), scales.fill(0.5)
    q, qa = act_array(rng, (1, 2, 64), "f32")
    L = cuda(np.array([n], np.int32))
    got = fb.page_select(q, cache, bounds, L, K, scale=1.0, first=0, last=2)
    assert got[0, 0].tolist() == E.select(qa[0], codes[table[0], 0], scales[table[0], 0], n, n, 1, 2, K, 1.0, 0, 2)
    for s in (1.0, -1.0):
        got = fb.page_select(q * 0, cache, bounds, L, K, scale=s, first=0, last=1)
        assert got[0, 0].tolist() == list(range(K - 1)) + [n - 1]


def test_page_select_with_invalid_pages_and_infinite_bounds(fb):
    rng = np.random.default_rng(4)
    n = 40
    cache, bounds, codes, scales, table = bounded_cache(fb, rng, n)
    q, _ = act_array(rng, (1, 1, 64), "f32")
    L = cuda(np.array([n], np.int32))
    bounds.scales[table[0, 33]] = float("inf")  # a score that is infinite or NaN counts as the largest
    got = fb.page_select(q, cache, bounds, L, 1, scale=1.0, first=0, last=0)
    assert got[0, 0].tolist() == [33] and fb.fa_back_get_error() == 0
    cache.page_table[0, 10:] = torch.tensor([-1, n, 10 ** 9] * 10, dtype=torch.int32, device="cuda")
    got = fb.page_select(q, cache, bounds, L, 12, scale=1.0, first=0, last=0)
    assert got[0, 0].tolist() == list(range(12))  # the ten that are there, then the lowest of the others
    assert fb.STATUS[fb.fa_back_get_error()] == "FA_ERR_PAGE"


# ------------------------------------------------------------------------------------------------
# attention over selected pages

def over_pages(p, pages, q, scale, softcap, alibi, sinks):
    """R.decode() of each KV head over the keys of its pages: O, lse, and what the tolerances scale with."""
    B, H, _ = q.shape
    G = H // p.Hkv
    O, lse, mag, smag = np.zeros((B, H, p.Dv)), np.full((B, H), -np.inf), np.zeros((B, H, p.Dv)), np.zeros((B, H))
    for b, L in enumerate(p.lens):
        for hk in range(p.Hkv):
            mine = [j for j in pages[b, hk] if 0 <= j < -(-max(L, 0) // p.page)]
            pos = np.concatenate([np.arange(j * p.page, min((j + 1) * p.page, L)) for j in mine] + [np.zeros(0, int)]).astype(int)
            for h in range(hk * G, (hk + 1) * G):
                every = np.zeros(0)
                if len(pos):
                    k, v, x64 = p.kd[b][pos, hk], p.vd[b][pos, hk], q[b, h].astype(np.float64)
                    x = scale * (k @ x64)
                    smag[b, h] = (abs(scale) * (np.abs(k) @ np.abs(x64))).max()
                    if softcap > 0:
                        x = softcap * np.tanh(x / softcap)
                    if alibi is not None:
                        x = x + float(alibi[h]) * (pos - (L - 1))
                        smag[b, h] += abs(float(alibi[h])) * L
                    every = x
                if sinks is not None:
                    every = np.append(every, float(sinks[h]))
                if len(every):
                    top = every.max()
                    lse[b, h] = top + np.log(np.exp(every - top).sum())
                if len(pos):
                    w = np.exp(x - lse[b, h])
                    O[b, h], mag[b, h] = w @ v, w @ np.abs(v)
                    smag[b, h] = max(smag[b, h], abs(lse[b, h]))
    return O, lse, mag, smag


SPARSE = {  # lens, H, Hkv, D, Dv, kt, vt, act, page, K, softcap, alibi, sinks
    "one_page": ((5,), 2, 1, 64, 64, "f16", "f16", "f32", 16, 1, 0.0, False, False),
    "q8": ((3000, 700, 0, 64, 1), 8, 2, 128, 128, "q8_0", "q8_0", "f32", 64, 9, 0.0, False, False),
    "ext_boxes_of_8": ((900, 40, 1000), 6, 3, 128, 64, "q4_0", "q8_0", "bf16", 40, 8, 20.0, True, True),
    "single_rows": ((333, 20, 5), 4, 2, 64, 128, "f32", "f16", "f16", 5, 21, 0.0, True, False),
    "single_rows_q4": ((333, 20, 5), 4, 1, 256, 64, "q4_0", "f16", "f32", 12, 11, 0.0, True, True),
    "many_heads": ((2000, 1999), 24, 2, 256, 256, "f16", "q4_0", "f32", 32, 20, 0.0, False, True),
    "page_of_one": ((70,), 2, 2, 64, 64, "f16", "f32", "f32", 1, 40, 0.0, False, False),
    "split": ((40000, 39990), 4, 1, 128, 128, "f16", "f16", "bf16", 128, 250, 0.0, True, False),
    "large_batch": (tuple(17 * i % 230 - 3 for i in range(300)), 4, 2, 64, 64, "q8_0", "f16", "f16", 16, 6, 0.0, False, False),
}


@pytest.mark.parametrize("name", sorted(SPARSE))
def test_paged_decode_pages(fb, name):
    """Random pages in any order, some of them none; the last, partly filled page somewhere among them."""
    lens, H, Hkv, D, Dv, kt, vt, act, page, K, softcap, alibi, sinks = SPARSE[name]
    p = R.Paged(len(name), lens, Hkv, D, Dv, TYPES[kt], TYPES[vt], page)
    rng = np.random.default_rng(len(name))
    B = len(lens)
    pages = np.full((B, Hkv, K), -1, np.int32)
    for b, L in enumerate(lens):
        n = -(-max(L, 0) // page)
        for hk in range(Hkv):
            m = min(K, n)
            mine = rng.permutation(n)[:m].astype(np.int32)
            if m:
                mine[rng.integers(0, m)] = n - 1 if n - 1 not in mine else mine[0] if m == 1 else -1
                if m > 3:
                    mine[rng.integers(0, m)] = [-1, n, 2 ** 31 - 1, -2 ** 31][rng.integers(0, 4)]
            seen, uniq = set(), []
            for j in mine.tolist():
                uniq.append(-1 if j in seen else j)
                seen.add(j)
            pages[b, hk, :m] = uniq
            pages[b, hk, m:] = rng.integers(0, max(n, 1), K - m)  # not read
    cache = p.on_gpu(fb, torch)
    q, qa = act_array(rng, (B, H, D), act)
    al = (2.0 ** -np.arange(2, H + 2)).astype(np.float32) if alibi else None
    sk = rng.standard_normal(H).astype(np.float32) if sinks else None
    scale = D ** -0.5
    got = fb.paged_decode(q, cache, cuda(np.array(lens, np.int32)), scale=scale, softcap=softcap, alibi_slopes=cuda(al), sinks=cuda(sk),
                          pages=cuda(pages))
    live = [b for b, L in enumerate(lens) if L >= 0]
    n_read = [[pages[b, hk, :min(K, -(-max(L, 0) // page))] for hk in range(Hkv)] for b, L in enumerate(lens)]
    O, lse, mag, smag = over_pages(p, {(b, hk): n_read[b][hk] for b in range(B) for hk in range(Hkv)}, qa, scale, softcap, al, sk)
    tol_O, tol_lse = R.decode_tolerance(p, mag, smag, act)
    within(got["O"].float().cpu().numpy()[live], O[live], tol_O[live] + half_step(act, O[live]), "O")
    within(got["lse"].cpu().numpy()[live], lse[live], tol_lse[live], "lse")
    assert fb.fa_back_get_error() == 0


@pytest.mark.parametrize("name", ["q8", "ext_boxes_of_8", "single_rows", "many_heads"])
def test_all_pages_is_the_plain_attention(fb, name):
    lens, H, Hkv, D, Dv, kt, vt, act, page, _, softcap, alibi, sinks = SPARSE[name]
    p = R.Paged(3, lens, Hkv, D, Dv, TYPES[kt], TYPES[vt], page)
    rng = np.random.default_rng(3)
    q, qa = act_array(rng, (len(lens), H, D), act)
    al, sk = (2.0 ** -np.arange(2, H + 2)).astype(np.float32), rng.standard_normal(H).astype(np.float32)
    kw = dict(scale=D ** -0.5, softcap=softcap, alibi_slopes=cuda(al) if alibi else None, sinks=cuda(sk) if sinks else None)
    cache, n = p.on_gpu(fb, torch), cuda(np.array(lens, np.int32))
    width = max(-(-L // page) for L in lens)
    every = torch.arange(width, dtype=torch.int32, device="cuda").expand(len(lens), Hkv, width).contiguous()
    one, two = fb.paged_decode(q, cache, n, **kw), fb.paged_decode(q, cache, n, pages=every, **kw)
    O, lse, mag, smag = R.decode(p, qa, D ** -0.5, softcap, al if alibi else None, sk if sinks else None)
    tol_O, tol_lse = R.decode_tolerance(p, mag, smag, act)
    for g in (one, two):
        within(g["O"].float().cpu().numpy(), O, tol_O + half_step(act, O), "O")
        within(g["lse"].cpu().numpy(), lse, tol_lse, "lse")


@pytest.mark.parametrize("page", [16, 8, 5])
def test_selected_pages_on_invalid_page_numbers_are_masked(fb, page):
    p = R.Paged(page, (200, 33), 2, 64, 64, 1, 0, page)
    cache, n = p.on_gpu(fb, torch), cuda(np.array([200, 33], np.int32))
    cache.page_table[0, 3], cache.page_table[1, 0] = -1, 10 ** 9
    pages = torch.tensor([[[0, 3, 4, 9, 12], [3, -1, -1, -1, -1]], [[0, 1, -1, -1, -1], [1, 0, -1, -1, -1]]], dtype=torch.int32, device="cuda")
    q, qa = act_array(np.random.default_rng(1), (2, 4, 64), "f32")
    got = fb.paged_decode(q, cache, n, scale=0.2, pages=pages)
    assert fb.STATUS[fb.fa_back_get_error()] == "FA_ERR_PAGE"
    left = {(0, 0): [0, 4, 9, 12], (0, 1): [], (1, 0): [1], (1, 1): [1]}
    O, lse, mag, smag = over_pages(p, left, qa, 0.2, 0.0, None, None)
    tol_O, tol_lse = R.decode_tolerance(p, mag, smag, "f32")
    within(got["O"].cpu().numpy(), O, tol_O), within(got["lse"].cpu().numpy(), lse, tol_lse)


def test_a_wait_that_runs_out_over_selected_pages(fb):
    """The limit that every wait counts as over: the error word says so, and the next call is right."""
    p = R.Paged(2, (300,), 2, 64, 64, 2, 2, 16)
    cache, n = p.on_gpu(fb, torch), cuda(np.array([300], np.int32))
    q, qa = act_array(np.random.default_rng(1), (1, 4, 64), "f32")
    pages = torch.arange(19, dtype=torch.int32, device="cuda").expand(1, 2, 19).contiguous()
    assert fb.fa_back_test_wait_limit(0) == 0
    fb.paged_decode(q, cache, n, scale=0.2, pages=pages)
    torch.cuda.synchronize()
    assert fb.STATUS[fb.fa_back_get_error()] == "FA_ERR_TIMEOUT"
    got, want = fb.paged_decode(q, cache, n, scale=0.2, pages=pages), R.decode(p, qa, 0.2)
    tol_O, _ = R.decode_tolerance(p, want[2], want[3], "f32")
    within(got["O"].cpu().numpy(), want[0], tol_O)
    assert fb.fa_back_get_error() == 0


def test_padding_slots_keep_their_rows(fb):
    p = R.Paged(1, (40, -1, 0), 1, 64, 64, 1, 1, 16)
    cache, n = p.on_gpu(fb, torch), cuda(np.array([40, -1, 0], np.int32))
    q = torch.randn(3, 2, 64, device="cuda")
    out = {"O": torch.full((3, 2, 64), 7.0, device="cuda"), "lse": torch.full((3, 2), 7.0, device="cuda")}
    pages = torch.full((3, 1, 2), -1, dtype=torch.int32, device="cuda")
    fb.paged_decode(q, cache, n, scale=1.0, pages=pages, out=out)
    assert (out["O"][1] == 7).all() and (out["lse"][1] == 7).all()
    assert not out["O"][[0, 2]].any() and torch.isneginf(out["lse"][[0, 2]]).all()  # no page, no key


# ------------------------------------------------------------------------------------------------
# together

def serve(fb, lists, cache, bounds, x, wq, wk, rope, axes, news, T, K, H, Hkv):
    """A step: room for the new tokens, the last of each request asks."""
    got = fb.pages_extend(lists, news, T)
    seq, pos = got["seq"], got["pos"]
    p = torch.stack([pos, pos // 7, pos % 7]).to(torch.int32)
    kw = dict(rope=rope, rope_axes=axes)
    fb.cache_append(x[:, H:H + Hkv], x[:, H + Hkv:], cache, seq, pos, k_norm=wk, rope_pos=p, **kw)
    fb.page_bounds(cache, bounds, lists.seq_lens, first=got["first"])
    q = fb.qk_norm_rope(x[:, :H], None, p, wq=wq, **kw)["q"]
    last = (got["starts"][1:].long() - 1).clamp_min(0)
    q = q[last].contiguous()
    pages = fb.page_select(q, cache, bounds, lists.seq_lens, K, scale=0.1, first=1, last=2)
    o = fb.paged_decode(q, cache, lists.seq_lens, scale=0.1, pages=pages)
    dense = fb.paged_decode(q, cache, lists.seq_lens, scale=0.1)
    return q, pages, o, dense


def test_steps_of_a_serving_loop(fb):
    """Prompts, decode steps, rejected drafts and requests that end and begin: every step's tables, slots, bounds,
    choice and attention against the definitions on a cache that is kept contiguous on the side."""
    rng = np.random.default_rng(8)
    gen = torch.Generator(device="cuda").manual_seed(8)
    B, H, Hkv, D, page, K = 5, 6, 2, 64, 8, 6
    lists = fb.PageLists.empty(B, 40, 150, page)
    raw = lambda t: torch.zeros(150, page, Hkv, fb.fa_row_bytes(t, D), dtype=torch.uint8, device="cuda")  # noqa: E731
    cache = fb.PagedCache(raw(fb.FA_Q8_0), fb.FA_Q8_0, raw(fb.FA_F16), fb.FA_F16, lists.page_table, D=D, Dv=D)
    bounds = fb.PageBounds.of(cache)
    wq, wk = (0.5 + torch.rand(D, generator=gen, device="cuda") for _ in range(2))
    rope, axes = fb.rope_frequencies(D), fb.rope_sections([16, 8, 8])
    lists.seq_lens.copy_(torch.tensor([0, 0, -1, 0, -1]))
    for step in range(6):
        news = [(100, 33, 0, 1, 0), (1, 1, 0, 1, 0), (4, 4, 0, 4, 0), (1, 1, 60, 1, 0), (1, 0, 1, 1, 0), (1, 1, 1, 1, 1)][step]
        T = sum(news) + 2
        x = torch.randn(T, H + 2 * Hkv, D, generator=gen, device="cuda").bfloat16()
        q, pages, o, dense = serve(fb, lists, cache, bounds, x, wq, wk, rope, axes, cuda(np.array(news, np.int32)), T, K, H, Hkv)
        lens = lists.seq_lens.tolist()
        p = R.Paged(0, [max(n, 0) for n in lens], Hkv, D, D, 2, 1, page)  # (only its fields are used)
        table = lists.page_table.cpu().numpy()
        kd, vd = [], []
        for n in lens:
            b = len(kd)
            j = torch.arange(max(n, 0), dtype=torch.int32, device="cuda")
            r = fb.cache_read(cache, torch.full_like(j, b), j)
            kd.append(r["k"].double().cpu().numpy()), vd.append(r["v"].double().cpu().numpy())
        p.kd, p.vd, p.table, p.lens = kd, vd, table, [max(n, 0) for n in lens]
        codes, scales = bounds.codes.cpu().numpy(), bounds.scales.cpu().numpy()
        for b, n in enumerate(p.lens):
            for i in range(-(-n // page)):
                c, s = want_bounds(p, b, i)
                assert np.array_equal(codes[table[b, i]], c) and np.array_equal(scales[table[b, i]], s), (step, b, i)
        live = [b for b, n in enumerate(lens) if n >= 0]
        sel = pages.cpu().numpy()
        qa = q.float().cpu().numpy()
        sel[[b for b in range(B) if b not in live]] = -77
        check_select(p, codes, scales, qa, sel, lens, H, K, 0.1, 1, 2)
        O, lse, mag, smag = over_pages(p, sel, qa, 0.1, 0.0, None, None)
        tol_O, tol_lse = R.decode_tolerance(p, mag, smag, "bf16")
        within(o["O"].float().cpu().numpy()[live], O[live], tol_O[live] + half_step("bf16", O[live]), "O")
        within(o["lse"].cpu().numpy()[live], lse[live], tol_lse[live], "lse")
        for b in live:  # a sequence of few pages: all of them are chosen
            if -(-lens[b] // page) <= K:
                within(o["lse"][b].cpu().numpy(), dense["lse"][b].double().cpu().numpy(), 2 * tol_lse[b])
        if step == 2:  # of four drafts one to four are taken; then a request ends and another begins
            keep = np.array([lens[0] - 3, lens[1] - 1, -1, lens[3], -1], np.int32)
            fb.pages_trim(lists, cuda(keep))
            lists.seq_lens[2] = 0
        if step == 4:
            fb.pages_trim(lists, cuda(np.array([-1, 0, -1, -1, -1], np.int32)))
            lists.seq_lens[4] = 0
    held = int((lists.page_table >= 0).sum())
    assert held + int(lists.num_free) == 150 and fb.fa_back_get_error() == 0


def test_a_captured_step_goes_on_with_what_it_finds(fb):
    """A decode step as a CUDA graph, replayed over growing requests: equal to eager steps on equal lists; a trim in a
    graph of its own gives up what a step has taken."""
    B, H, Hkv, D, page, K = 4, 4, 2, 128, 16, 3
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(9, B, H + 2 * Hkv, D, generator=gen, device="cuda").half()
    rope, axes = fb.rope_frequencies(D), fb.rope_sections([16, 24, 24], interleaved=True)
    w = 0.5 + torch.rand(D, generator=gen, device="cuda")
    news = torch.ones(B, dtype=torch.int32, device="cuda")

    def world():
        lists = fb.PageLists.empty(B, 10, 60, page)
        raw = torch.zeros(60, page, Hkv, fb.fa_row_bytes(fb.FA_Q4_0, D), dtype=torch.uint8, device="cuda")
        cache = fb.PagedCache(raw, fb.FA_Q4_0, raw.clone(), fb.FA_Q4_0, lists.page_table, D=D, Dv=D)
        lists.seq_lens.copy_(torch.tensor([0, 0, 0, -1]))
        return lists, cache, fb.PageBounds.of(cache)

    def step(wd, xs):
        return serve(fb, *wd, xs, w, w, rope, axes, news, B, K, H, Hkv)

    a, b = world(), world()
    xs = x[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(b, xs)  # (warm-up)
        fb.pages_trim(b[0], torch.zeros_like(news))
    torch.cuda.current_stream().wait_stream(side)
    graph, undo = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    keep = b[0].seq_lens.clone()
    with torch.cuda.graph(graph):
        got = step(b, xs)
    with torch.cuda.graph(undo):
        fb.pages_trim(b[0], keep)
    for i in range(9):
        want = step(a, x[i])
        xs.copy_(x[i])
        keep.copy_(b[0].seq_lens)
        graph.replay()
        if i % 4 == 3:
            undo.replay()
            assert torch.equal(b[0].seq_lens, keep)
            graph.replay()
        for t in ("page_table", "seq_lens", "free", "num_free"):
            assert torch.equal(getattr(a[0], t), getattr(b[0], t)), (i, t)
        assert torch.equal(a[1].k, b[1].k)
        assert torch.equal(want[1][:3], got[1][:3]) and torch.equal(want[2]["O"][:3], got[2]["O"][:3])
    assert fb.fa_back_get_error() == 0


def test_calls_on_another_stream(fb):
    p = R.Paged(6, (500, 300), 2, 64, 64, 2, 2, 16)
    cache, n = p.on_gpu(fb, torch), cuda(np.array([500, 300], np.int32))
    q = torch.randn(2, 4, 64, device="cuda")
    one, two = fb.PageBounds.of(cache), fb.PageBounds.of(cache)
    fb.page_bounds(cache, one, n)
    pages = fb.page_select(q, cache, one, n, 5, scale=1.0)
    o = fb.paged_decode(q, cache, n, scale=1.0, pages=pages)
    la, lb = (lists_of(fb, np.random.default_rng(1), 30, 6, 100, 16, 0.3)[0] for _ in range(2))
    news = torch.full((30,), 3, dtype=torch.int32, device="cuda")
    keep = la.seq_lens.clone()
    e = fb.pages_extend(la, news, 90)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    fb.page_bounds(cache, two, n, stream=s)
    ws = fb.Workspace()
    pages2 = fb.page_select(q, cache, two, n, 5, scale=1.0, workspace=ws, stream=s)
    o2 = fb.paged_decode(q, cache, n, scale=1.0, pages=pages2, stream=s)
    e2 = fb.pages_extend(lb, news, 90, stream=s)
    s.synchronize()
    assert torch.equal(one.codes, two.codes) and torch.equal(one.scales, two.scales) and torch.equal(pages, pages2)
    assert torch.equal(o["O"], o2["O"]) and torch.equal(o["lse"], o2["lse"]) and all(torch.equal(e[k], e2[k]) for k in e)
    fb.pages_trim(lb, keep, stream=s)
    s.synchronize()
    assert torch.equal(lb.seq_lens, keep)


def test_the_marshalling_module_and_python_make_the_same_calls(fb, monkeypatch):
    from flash_attention_backward_gb300 import paged
    assert paged._fast is not None
    p = R.Paged(5, (200, 90, 33), 2, 128, 128, 2, 3, 16)
    cache, n = p.on_gpu(fb, torch), cuda(np.array([200, 90, 33], np.int32))
    x = torch.randn(3, 8, 128, device="cuda").bfloat16()
    w = torch.rand(128, device="cuda")
    p3 = cuda(np.arange(9, dtype=np.int32).reshape(3, 3))
    kw = dict(rope=fb.rope_frequencies(64), rope_axes=fb.rope_sections([8, 16, 8]))
    seq, pos = cuda(np.array([0, 1, 2], np.int32)), cuda(np.array([5, 6, 7], np.int32))
    news = cuda(np.array([20, 0, 3], np.int32))

    def every():
        lists = lists_of(fb, np.random.default_rng(2), 3, 9, 30, 16, 0.5)[0]
        keep = lists.seq_lens.clone()
        out = [fb.pages_extend(lists, news, 23), {"lens": lists.seq_lens.clone()}]
        fb.pages_trim(lists, keep)
        bounds = fb.PageBounds.of(cache)
        fb.page_bounds(cache, bounds, n)
        fb.page_bounds(cache, bounds, n, first=pos)
        pages = fb.page_select(x[:, :6], cache, bounds, n, 4, scale=0.5, first=0, last=1, alibi_slopes=w[:6].contiguous())
        out += [{"pages": pages, "codes": bounds.codes, "scales": bounds.scales, "free": lists.free},
                fb.paged_decode(x[:, :6], cache, n, scale=0.5, pages=pages),
                fb.qk_norm_rope(x[:, :6], x[:, 6:], p3, wq=w, wk=w, **kw),
                fb.qk_norm_rope_backward(x[:, :6].contiguous(), None, x[:, :6], None, p3, wq=w, **kw)]
        fb.cache_append(x[:, :2], x[:, 2:4], cache, seq, pos, k_norm=w, rope_pos=p3, **kw)
        return out + [{"k": cache.k.clone(), "v": cache.v.clone()}]

    reached = []
    real = paged._call
    monkeypatch.setattr(paged, "_call", lambda *a: reached.append(1) or real(*a))
    from flash_attention_backward_gb300 import pages as pages_mod
    monkeypatch.setattr(pages_mod, "_call", lambda *a: reached.append(1) or real(*a))
    fast = every()
    assert not reached  # all of them by the module
    monkeypatch.setattr(paged, "_fast", None)
    monkeypatch.setattr(paged, "_plain", False)
    cache.k.copy_(torch.from_numpy(p.k)), cache.v.copy_(torch.from_numpy(p.v))
    slow = every()
    assert len(reached) == 9
    for f, g in zip(fast, slow):
        assert list(f) == list(g)
        for k in f:
            assert torch.equal(f[k], g[k]), k
