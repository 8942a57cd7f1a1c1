"""The paged-cache and norm / rotation operators on the GPU, against 64-bit numpy (tests/paged_ref.py).

Tolerances are bounds from the roundings that each operator makes, written beside them; the result's
own rounding to a 16-bit type adds half a step of that type.
"""
import numpy as np
import pytest

import paged_ref as R
import synth

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, F16, Q8, Q4 = 0, 1, 2, 3
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def fb():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import flash_attention_backward_gb300 as m
    from flash_attention_backward_gb300 import build
    build.build()
    return m


def half_step(act, ref):
    return 0.0 if act == "f32" else torch.finfo(DT[act]).eps / 2 * np.abs(ref) * 1.01 + torch.finfo(DT[act]).smallest_normal * 2.0 ** -8


def act_array(rng, shape, act):
    """Seeded normals rounded to the activation type: the tensor and its exact values."""
    t = torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(DT[act]).cuda()
    return t, t.float().cpu().numpy()


def within(got, ref, tol, what=""):
    got = np.asarray(got, np.float64)
    fin = np.isfinite(ref)
    assert np.array_equal(np.isneginf(got), np.isneginf(ref)), what
    off, tol = np.abs(got[fin] - ref[fin]), np.broadcast_to(tol, ref.shape)[fin]
    bad = ~(off <= tol)
    assert not bad.any(), (what, int(bad.sum()), off[bad][:4], tol[bad][:4])


# ------------------------------------------------------------------------------------------------
# norm and rotation

NORM = {  # N, H, Hkv, D, act, out, n_rot, halves, weights, fused
    "one_token": (1, 1, 1, 64, "f32", "f32", 64, True, True, False),
    "odd": (37, 6, 2, 128, "f32", "f32", 128, True, True, False),
    "d256_bf16": (19, 5, 5, 256, "bf16", "bf16", 256, True, True, False),
    "partial_halves": (33, 4, 1, 64, "f16", "f32", 16, True, True, True),
    "partial_pairs": (33, 4, 3, 128, "bf16", "f16", 34, False, True, True),
    "pairs": (50, 3, 1, 64, "f32", "bf16", 64, False, True, False),
    "no_norm": (21, 4, 2, 128, "f32", "f32", 64, True, False, False),
    "no_rotation": (21, 4, 2, 256, "f16", "f16", 0, True, True, True),
    "many_tokens": (1500, 9, 3, 64, "bf16", "f32", 64, True, True, True),
    "queries_only": (40, 7, 0, 128, "f32", "f32", 128, False, True, False),
}


def norm_inputs(name):
    N, H, Hkv, D, act, out, n_rot, halves, weights, fused = NORM[name]
    rng = np.random.default_rng(sorted(NORM).index(name) + 100)
    if fused:  # one projection, with columns that belong to neither tensor
        x, xa = act_array(rng, (N, H + 2 * Hkv + 1, D), act)
        q, k, qa, ka = x[:, :H], x[:, H:H + Hkv], xa[:, :H], xa[:, H:H + Hkv]
    else:
        (q, qa), (k, ka) = act_array(rng, (N, H, D), act), act_array(rng, (N, Hkv, D), act)
    pos = rng.integers(-5, 2000000, N).astype(np.int32)
    w = [(1.0 + 0.2 * rng.standard_normal(D)).astype(np.float32) if weights else None for _ in range(2)]
    return (N, H, Hkv, D, act, out, n_rot, halves), q, k, qa, ka, pos, w, rng


def cuda(a):
    return None if a is None else torch.from_numpy(a).cuda()


@pytest.mark.parametrize("name", sorted(NORM))
def test_norm_rope(fb, name):
    (N, H, Hkv, D, act, out, n_rot, halves), q, k, qa, ka, pos, w, _ = norm_inputs(name)
    rope = fb.rope_frequencies(n_rot, 10000.0) if n_rot else None
    got = fb.qk_norm_rope(q, k if Hkv else None, cuda(pos), wq=cuda(w[0]), wk=cuda(w[1]) if Hkv else None, eps=1e-6, rope=rope,
                          rope_style=int(halves), dtype=DT[out])
    for n, x, wt in (("q", qa, w[0]), ("k", ka, w[1])):
        if not x.shape[1]:
            assert got[n] is None
            continue
        y = R.norm(x, wt, 1e-6) if wt is not None else x.astype(np.float64)
        ref = R.rotate(y, pos, n_rot, 10000.0, halves) if n_rot else y
        # r: sum of squares in chains of 8 and 5 (13 u, halved), its root 2 u, two products; cos and sin
        # within 3 u and the 32-bit angle's float rounding (pi 2^-25 < 2 u): under 20 u of the pair's magnitude
        mag = np.abs(y)
        if n_rot:
            i = np.arange(n_rot // 2)
            f, s = (i, i + n_rot // 2) if halves else (2 * i, 2 * i + 1)
            pair = mag[..., f] + mag[..., s]
            mag = mag.copy()
            mag[..., f] = mag[..., s] = pair
        within(got[n].float().cpu().numpy(), ref, 20 * U * mag + half_step(out, ref), n)
    assert fb.fa_back_get_error() == 0


def back_reference(x, w, gy, pos, n_rot, halves, eps=1e-6):
    """dx, dw and the magnitudes that their roundings scale with."""
    x, gy = x.astype(np.float64), gy.astype(np.float64)
    g = R.rotate(gy, pos, n_rot, 10000.0, halves, -1.0) if n_rot else gy
    if w is None:
        return g, None, None, None, g
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    h = g * w.astype(np.float64)
    dx = r * (h - x * r * r * (h * x).mean(-1, keepdims=True))
    return dx, (g * x * r).sum((0, 1)), r, h, g


@pytest.mark.parametrize("name", sorted(NORM))
def test_norm_rope_backward(fb, name):
    (N, H, Hkv, D, act, out, n_rot, halves), q, k, qa, ka, pos, w, rng = norm_inputs(name)
    (gq, gqa), (gk, gka) = act_array(rng, (N, H, D), out), act_array(rng, (N, Hkv, D), out)
    rope = fb.rope_frequencies(n_rot, 10000.0) if n_rot else None
    got = fb.qk_norm_rope_backward(gq, gk if Hkv else None, q, k if Hkv else None, cuda(pos), wq=cuda(w[0]),
                                   wk=cuda(w[1]) if Hkv else None, eps=1e-6, rope=rope, rope_style=int(halves))
    for n, x, wt, gy in (("q", qa, w[0], gqa), ("k", ka, w[1], gka)):
        if not x.shape[1]:
            assert "d" + n not in got
            continue
        dx, dw, r, h, g = back_reference(x, wt, gy, pos, n_rot, halves)
        gmax = np.abs(g).max(-1, keepdims=True) + np.abs(gy).max(-1, keepdims=True)
        if wt is None:
            within(got["d" + n].float().cpu().numpy(), dx, 20 * U * gmax + half_step(act, dx), "d" + n)
            assert "dw" + n not in got
            continue
        # as the forward's, twice (g, then the product with r), and the mean of h o x: 20 u of its magnitudes
        x64, wm = x.astype(np.float64), np.abs(wt).max()
        mag = r * (gmax * wm + np.abs(x64) * r * r * (gmax * wm * np.abs(x64)).mean(-1, keepdims=True))
        within(got["d" + n].float().cpu().numpy(), dx, 48 * U * mag + half_step(act, dx), "d" + n)
        # dw: terms within 40 u of theirs, summed in chains of at most rows / 8 + 400 additions
        terms = (gmax * np.abs(x64) * r).sum((0, 1))
        rows = N * x.shape[1]
        within(got["dw" + n].cpu().numpy(), dw, (40 + rows / 8 + 400) * U * terms, "dw" + n)
    assert fb.fa_back_get_error() == 0


def test_norm_rope_backward_against_differences(fb):
    """<dx, v> + <dw, u> is the central difference of <gy, y> along (v, u), taken in 64 bits."""
    rng = np.random.default_rng(7)
    N, H, Hkv, D = 9, 4, 2, 64
    (q, qa), (k, ka), (gq, gqa), (gk, gka) = (act_array(rng, (N, h, D), "f32") for h in (H, Hkv, H, Hkv))
    pos = rng.integers(0, 100000, N).astype(np.int32)
    w = [(1.0 + 0.2 * rng.standard_normal(D)).astype(np.float32) for _ in range(2)]
    rope = fb.rope_frequencies(32, 10000.0)
    got = fb.qk_norm_rope_backward(gq, gk, q, k, cuda(pos), wq=cuda(w[0]), wk=cuda(w[1]), rope=rope, rope_style=fb.FA_ROPE_HALVES)
    for n, x, wt, gy in (("q", qa, w[0], gqa), ("k", ka, w[1], gka)):
        v, uw, e = rng.standard_normal(x.shape), rng.standard_normal(D), 1e-5
        x, wt, gy = (a.astype(np.float64) for a in (x, wt, gy))
        f = lambda t: (gy * R.rotate(R.norm(x + t * v, wt + t * uw, 1e-6), pos, 32, 10000.0, True)).sum()  # noqa: E731
        num = (f(e) - f(-e)) / (2 * e)
        dx, dw = got["d" + n].double().cpu().numpy(), got["dw" + n].double().cpu().numpy()
        ana = (dx * v).sum() + (dw * uw).sum()
        scale = np.sqrt((dx ** 2).sum() * (v ** 2).sum())
        assert abs(num - ana) <= 1e-5 * scale, (n, num, ana)  # differences: e^2 and 1e-16 / e; the gradients: some u


def test_norm_rope_in_place_and_same_input_twice(fb):
    rng = np.random.default_rng(3)
    q, _ = act_array(rng, (65, 5, 128), "bf16")
    w, pos = torch.rand(128, device="cuda") + 0.5, torch.arange(65, dtype=torch.int32, device="cuda")
    rope = fb.rope_frequencies(128, 10000.0)
    ref = fb.qk_norm_rope(q, q, pos, wq=w, wk=w, rope=rope)
    assert torch.equal(ref["q"], ref["k"])
    k = q.clone()
    got = fb.qk_norm_rope(q, k, pos, wq=w, wk=w, rope=rope, out={"q": q, "k": k})
    assert got["q"] is q and torch.equal(q, ref["q"]) and torch.equal(k, ref["k"])


@pytest.mark.parametrize("layout", ["interleaved", "odd_rows", "broadcast"])
def test_norm_rope_layouts(fb, layout):
    """Heads apart from each other, rows that start off 16 bytes, one token's heads for every token: the same
    results as from contiguous copies, both ways."""
    rng = np.random.default_rng(12)
    N, H, Hkv, D = 53, 13, 3, 128
    if layout == "interleaved":  # [N][Hkv][q .. q, k, v] as some projections have them
        x, _ = act_array(rng, (N, Hkv, 6, D), "bf16")
        q, k = x[:, :, 0], x[:, :, 4]
    elif layout == "odd_rows":
        flat, _ = act_array(rng, (N * (H + Hkv) * D + 3,), "bf16")
        x = flat[3:].view(N, H + Hkv, D)
        q, k = x[:, :H], x[:, H:]
    else:
        (q, _), (k, _) = act_array(rng, (1, H, D), "bf16"), act_array(rng, (N, 1, D), "bf16")
        q, k = q.expand(N, H, D), k.expand(N, Hkv, D)
    w, rope = torch.rand(D, device="cuda") + 0.5, fb.rope_frequencies(D)
    pos = torch.arange(N, dtype=torch.int32, device="cuda") * 7
    gq, gk = torch.randn(q.shape, device="cuda"), torch.randn(k.shape, device="cuda")
    for style in (fb.FA_ROPE_HALVES, fb.FA_ROPE_PAIRS):
        kw = dict(wq=w, wk=w, rope=rope, rope_style=style)
        a, b = (fb.qk_norm_rope(x, y, pos, **kw) for x, y in ((q, k), (q.contiguous(), k.contiguous())))
        for n in ("q", "k"):
            assert torch.equal(a[n], b[n])
        a, b = (fb.qk_norm_rope_backward(gq, gk, x, y, pos, **kw) for x, y in ((q, k), (q.contiguous(), k.contiguous())))
        for n in ("dq", "dk"):
            assert torch.equal(a[n], b[n])
        for n in ("dwq", "dwk"):  # (other runs of rows: another order of the sum)
            assert float((a[n] - b[n]).abs().max()) <= 1e-4 * float(b[n].abs().max())


def test_norm_rope_many_heads_and_rows(fb):
    """More heads than a warp takes at a time, and tokens that do not divide into the warps' runs."""
    rng = np.random.default_rng(13)
    for N, H, Hkv, D, act in ((3, 131, 67, 64, "f16"), (2501, 5, 1, 256, "bf16"), (1, 40, 8, 128, "f32"), (9000, 1, 1, 64, "f32")):
        (q, qa), (k, ka), (gq, gqa), (gk, gka) = (act_array(rng, (N, h, D), act) for h in (H, Hkv, H, Hkv))
        pos = rng.integers(0, 1 << 20, N).astype(np.int32)
        w = [(1.0 + 0.2 * rng.standard_normal(D)).astype(np.float32) for _ in range(2)]
        kw = dict(wq=cuda(w[0]), wk=cuda(w[1]), rope=fb.rope_frequencies(D // 2))
        y = fb.qk_norm_rope(q, k, cuda(pos), dtype=torch.float32, **kw)
        g = fb.qk_norm_rope_backward(gq, gk, q, k, cuda(pos), **kw)
        for n, x, wt, gy in (("q", qa, w[0], gqa), ("k", ka, w[1], gka)):
            ref = R.rotate(R.norm(x, wt, 1e-6), pos, D // 2, 10000.0, True)
            dx, dw, *_ = back_reference(x, wt, gy, pos, D // 2, True)
            for got, want, tol in ((y[n], ref, 1e-6), (g["d" + n], dx, 1e-6 if act == "f32" else 3e-3), (g["dw" + n], dw, 1e-5)):
                e = got.double().cpu().numpy() - want  # (rms: 2^-8.5 / sqrt 3 of bf16's own rounding, some 2^-24 otherwise)
                assert (e ** 2).sum() <= tol ** 2 * (want ** 2).sum(), (N, n)
    assert fb.fa_back_get_error() == 0


def test_norm_rope_backward_is_deterministic_and_empty(fb):
    rng = np.random.default_rng(4)
    (q, _), (g, _) = act_array(rng, (700, 6, 64), "f32"), act_array(rng, (700, 6, 64), "f32")
    w = torch.rand(64, device="cuda") + 0.5
    a, b = (fb.qk_norm_rope_backward(g, None, q, None, None, wq=w) for _ in range(2))
    assert torch.equal(a["dwq"], b["dwq"]) and torch.equal(a["dq"], b["dq"])
    e = fb.qk_norm_rope_backward(g[:0], None, q[:0], None, None, wq=w)
    assert e["dq"].shape == (0, 6, 64) and torch.equal(e["dwq"], torch.zeros(64, device="cuda"))


# ------------------------------------------------------------------------------------------------
# append and read

def empty_cache(fb, B, max_pages, page, Hkv, D, Dv, kt, vt, seed=0, fill=0xA5):
    n = B * max_pages + 2
    table = np.random.default_rng(seed).permutation(n)[: B * max_pages].reshape(B, max_pages).astype(np.int32)
    k = torch.full((n, page, Hkv, synth.row_bytes(kt, D)), fill, dtype=torch.uint8, device="cuda")
    v = torch.full((n, page, Hkv, synth.row_bytes(vt, Dv)), fill, dtype=torch.uint8, device="cuda")
    return fb.PagedCache(k, kt, v, vt, torch.from_numpy(table).cuda(), D=D, Dv=Dv), table


def rows_of(table, seq, pos, page):
    return table[seq, pos // page], pos % page


APPEND = {  # T, B, Hkv, D, Dv, kt, vt, act, page, n_rot, halves, k_norm
    "one": (1, 1, 1, 64, 64, Q8, Q8, "f32", 16, 64, True, True),
    "q8_q4": (77, 5, 2, 128, 128, Q8, Q4, "bf16", 16, 128, True, True),
    "q4_q8_d256": (50, 3, 4, 256, 256, Q4, Q8, "f32", 40, 64, False, False),
    "f16_f32": (61, 4, 3, 64, 128, F16, F32, "f16", 4, 16, True, False),
    "f32_f16": (200, 2, 1, 256, 64, F32, F16, "bf16", 7, 256, False, True),
    "q8_q8_many": (3001, 9, 8, 128, 128, Q8, Q8, "f16", 64, 128, True, True),
    "q4_q4_small": (33, 33, 1, 64, 64, Q4, Q4, "f32", 4, 64, True, True),
    "q8_plain": (40, 2, 2, 64, 256, Q8, Q8, "bf16", 8, 0, True, False),
}


@pytest.mark.parametrize("name", sorted(APPEND))
def test_append_and_read(fb, name):
    T, B, Hkv, D, Dv, kt, vt, act, page, n_rot, halves, k_norm = APPEND[name]
    rng = np.random.default_rng(sorted(APPEND).index(name) + 50)
    max_pages = -(-(T + 20) // page)
    cache, table = empty_cache(fb, B, max_pages, page, Hkv, D, Dv, kt, vt, seed=T)
    seq = rng.integers(0, B, T).astype(np.int32)
    pos = np.zeros(T, np.int32)
    for b in range(B):  # distinct rows, in no order
        pos[seq == b] = rng.permutation(T + 20)[: (seq == b).sum()]
    pad = rng.random(T) < 0.1 if T > 1 else np.zeros(T, bool)
    seq_in = np.where(pad & (np.arange(T) % 2 == 0), -1, seq).astype(np.int32)
    pos_in = np.where(pad & (np.arange(T) % 2 == 1), -1, pos).astype(np.int32)
    (k, ka), (v, va) = act_array(rng, (T, Hkv, D), act), act_array(rng, (T, Hkv, Dv), act)
    va[0, 0, :32] = 0.0  # a block of zeros
    v[0, 0, :32] = 0.0
    w = (1.0 + 0.2 * rng.standard_normal(D)).astype(np.float32) if k_norm else None
    rope = fb.rope_frequencies(n_rot, 10000.0) if n_rot else None
    before = cache.k.clone(), cache.v.clone()
    fb.cache_append(k, v, cache, cuda(seq_in), cuda(pos_in), k_norm=cuda(w), rope=rope, rope_style=int(halves))
    torch.cuda.synchronize()
    assert fb.fa_back_get_error() == 0

    live = ~pad
    at = rows_of(table, seq[live], pos[live], page)
    kraw, vraw = cache.k.cpu().numpy()[at], cache.v.cpu().numpy()[at]
    # every other row is left as it was
    for pool, old in ((cache.k, before[0]), (cache.v, before[1])):
        keep = torch.ones(pool.shape[:2], dtype=torch.bool, device="cuda")
        keep[torch.from_numpy(at[0]).cuda().long(), torch.from_numpy(at[1]).cuda().long()] = False
        assert torch.equal(pool[keep], old[keep])

    # values are stored from exact inputs: the same codes and scales as the definition's, bit for bit
    n = int(live.sum())
    vdec = R.oracle.dequant(vraw, vt, Dv).reshape(n, Hkv, Dv)
    assert np.array_equal(vdec, R.stored(va[live].astype(np.float64), vt)[1])
    # keys carry the norm's and rotation's f32 roundings (20 u of the pair, see above); where that crosses
    # a border between two codes or two f16 values, the stored value is the neighbouring one
    y = R.norm(ka, w, 1e-6) if k_norm else ka.astype(np.float64)
    mag = np.abs(y).max(-1, keepdims=True)
    if n_rot:
        y = R.rotate(y, pos, n_rot, 10000.0, halves)
    y, mag = y[live], 2 * mag[live]
    kdec = R.oracle.dequant(kraw, kt, D).reshape(n, Hkv, D)
    if kt == F32:
        step = 0.0
    elif kt == F16:
        step = 2.0 ** -10 * np.abs(y) + 2.0 ** -24
    else:
        amax = np.abs(y.reshape(n, Hkv, D // 32, 32)).max(-1, keepdims=True)
        step = np.broadcast_to(amax / (127 if kt == Q8 else 8) * 1.001, (n, Hkv, D // 32, 32)).reshape(y.shape)
    ref = R.stored(y, kt)[1]
    scale = 2.0 ** -10 if kt in (Q8, Q4) else 0.0  # the binary16 scale may be the neighbouring one too
    within(kdec, ref, step * 1.001 + 20 * U * mag + scale * np.abs(ref), "k")
    if kt != F32:  # borders are rare: nearly all rows agree to the f32 roundings
        assert np.mean(np.abs(kdec - ref) > 20 * U * mag + 1e-30) < 2e-3

    # read: decoded in every type, rows of skipped tokens left alone, and raw
    for rd in ("f32", "f16", "bf16"):
        out = {"k": torch.full((T, Hkv, D), 7.0, dtype=DT[rd], device="cuda"), "v": torch.full((T, Hkv, Dv), 7.0, dtype=DT[rd], device="cuda")}
        fb.cache_read(cache, cuda(seq_in), cuda(pos_in), dtype=DT[rd], out=out)
        for x, dec in (("k", kdec), ("v", vdec)):
            g = out[x].cpu()
            assert torch.equal(g[torch.from_numpy(live)], torch.from_numpy(dec).float().to(DT[rd])), (x, rd)
            assert bool((g[torch.from_numpy(pad)] == 7.0).all())
    raw = fb.cache_read(cache, cuda(seq[live]), cuda(pos[live]), dtype=torch.uint8)
    assert np.array_equal(raw["k"].cpu().numpy(), kraw) and np.array_equal(raw["v"].cpu().numpy(), vraw)
    assert fb.fa_back_get_error() == 0


def test_quantisers_on_borders_and_extremes(fb):
    """Values on and beside the borders between codes, ties of the largest magnitude, tiny and zero blocks."""
    Hkv, D = 1, 64
    rows = []
    for top in (127.0, 1.0, 3.0, 254.0, 2.0 ** -10, 1e-12, 0.0):
        n = np.arange(32)
        for shift in (0.0, 2.0 ** -22, -(2.0 ** -22)):
            blk = (n - 15.5) * top / 31.0 * (1.0 + shift)
            half = np.clip((n - 16) + 0.5, -126.5, 126.5) * top / 127.0 * (1.0 + shift)
            blk[3], half[5] = top, -top
            rows += [np.concatenate([blk, half])]
    sign = np.where(np.arange(64) % 2, -1.0, 1.0)
    rows += [sign * 5.0, -sign * 5.0, np.r_[np.full(32, -2.0), np.full(32, 2.0)], sign * (np.arange(64) % 32 + 1) / 32]
    x = np.stack(rows)[:, None, :].astype(np.float32)
    T = x.shape[0]
    for act in ("f32", "bf16"):
        t = cuda(x).to(DT[act])
        for ty in (Q8, Q4):
            cache, table = empty_cache(fb, 1, -(-T // 16), 16, Hkv, D, D, ty, ty)
            seq, pos = np.zeros(T, np.int32), np.arange(T, dtype=np.int32)
            fb.cache_append(t, t, cache, cuda(seq), cuda(pos))
            got = fb.cache_read(cache, cuda(seq), cuda(pos))
            ref = R.stored(t.float().cpu().numpy().astype(np.float64), ty)[1]
            for n in ("k", "v"):
                assert np.array_equal(got[n].cpu().numpy().astype(np.float64), ref.astype(np.float32).astype(np.float64)), (act, ty, n)


@pytest.mark.parametrize("seed", range(10))
def test_append_random(fb, seed):
    """Seeded random shapes: values bit for bit, keys without norm and rotation too, unwritten rows untouched."""
    r = np.random.default_rng(7000 + seed)
    pick = lambda *a: a[int(r.integers(len(a)))]  # noqa: E731
    D, Dv, Hkv = pick(64, 128, 256), pick(64, 128, 256), pick(1, 2, 3, 5, 8, 16)
    kt, vt, act, page = pick(F32, F16, Q8, Q4), pick(F32, F16, Q8, Q4), pick("f32", "f16", "bf16"), pick(16, 20, 64)
    T, B = int(np.exp(r.uniform(0, np.log(900)))), int(r.integers(1, 6))
    cache, table = empty_cache(fb, B, -(-T // page) + 1, page, Hkv, D, Dv, kt, vt, seed=seed)
    seq = r.integers(0, B, T).astype(np.int32)
    pos = np.array([(seq[:t] == seq[t]).sum() for t in range(T)], np.int32)
    (k, ka), (v, va) = act_array(r, (T, Hkv, D), act), act_array(r, (T, Hkv, Dv), act)
    fb.cache_append(k, v, cache, cuda(seq), cuda(pos))
    raw = fb.cache_read(cache, cuda(seq), cuda(pos), dtype=torch.uint8)
    dec = fb.cache_read(cache, cuda(seq), cuda(pos))
    for n, x, ty, d in (("k", ka, kt, D), ("v", va, vt, Dv)):
        ref = R.stored(x.astype(np.float64), ty)[1]
        got = R.oracle.dequant(raw[n].cpu().numpy(), ty, d).reshape(ref.shape)
        assert np.array_equal(got, ref), n
        assert np.array_equal(dec[n].cpu().numpy().astype(np.float64), ref.astype(np.float32).astype(np.float64)), n
        pool = cache.k if n == "k" else cache.v
        untouched = np.ones(pool.shape[:2], bool)
        untouched[rows_of(table, seq, pos, page)] = False
        assert bool((pool.cpu()[torch.from_numpy(untouched)] == 0xA5).all())
    assert fb.fa_back_get_error() == 0


@pytest.mark.parametrize("ty", [Q8, Q4])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf, 1e9])
@pytest.mark.parametrize("at", [0, 13, 31])
def test_append_block_without_a_finite_scale(fb, ty, bad, at):
    """A block that holds a NaN, an infinity or a value beyond binary16's scale decodes to no finite value;
    the blocks beside it are as they would be."""
    rng = np.random.default_rng(at)
    x = rng.standard_normal((2, 1, 64)).astype(np.float32)
    x[1, 0, 32 + at] = bad
    cache, _ = empty_cache(fb, 1, 1, 16, 1, 64, 64, ty, ty)
    seq, pos = cuda(np.zeros(2, np.int32)), cuda(np.arange(2, dtype=np.int32))
    fb.cache_append(cuda(x), cuda(x), cache, seq, pos)
    got = fb.cache_read(cache, seq, pos)
    clean = x.copy()
    clean[1, 0, 32:] = 0.0
    ref = R.stored(clean.astype(np.float64), ty)[1].astype(np.float32)
    for n in ("k", "v"):
        g = got[n].cpu().numpy()
        assert not np.isfinite(g[1, 0, 32:]).any()
        assert np.array_equal(g[0], ref[0]) and np.array_equal(g[1, 0, :32], ref[1, 0, :32])


def test_append_strided_views_match_contiguous(fb):
    rng = np.random.default_rng(11)
    T, H, Hkv, D = 45, 4, 2, 128
    x, _ = act_array(rng, (T, H + 2 * Hkv, D), "bf16")
    seq, pos = torch.zeros(T, dtype=torch.int32, device="cuda"), torch.arange(T, dtype=torch.int32, device="cuda")
    rope = fb.rope_frequencies(D)
    odd = torch.empty(T * (H + 2 * Hkv) * D + 1, dtype=torch.bfloat16, device="cuda")[1:].view_as(x)  # rows off 16 bytes
    odd.copy_(x)
    pools = []
    for kk, vv in ((x[:, H:H + Hkv], x[:, H + Hkv:]), (x[:, H:H + Hkv].contiguous(), x[:, H + Hkv:].contiguous()),
                   (odd[:, H:H + Hkv], odd[:, H + Hkv:])):
        cache, _ = empty_cache(fb, 1, 3, 16, Hkv, D, D, Q8, Q4)
        fb.cache_append(kk, vv, cache, seq, pos, rope=rope)
        pools.append((cache.k, cache.v))
    for a in pools[1:]:
        assert torch.equal(a[0], pools[0][0]) and torch.equal(a[1], pools[0][1])


def test_invalid_pages_sequences_and_positions_are_reported_and_skipped(fb):
    cache, table = empty_cache(fb, 2, 2, 16, 1, 64, 64, F16, F16)
    cache.page_table[1, 1] = 99
    cache.page_table[0, 1] = -7
    x = torch.ones(5, 1, 64, device="cuda")
    before = cache.k.clone()
    seq, pos = cuda(np.array([0, 1, 2, 0, 1], np.int32)), cuda(np.array([3, 17, 0, 16, 32], np.int32))
    fb.cache_append(x, x, cache, seq, pos)
    torch.cuda.synchronize()
    assert fb.STATUS[fb.fa_back_get_error()] == "FA_ERR_PAGE" and fb.fa_back_get_error() == 0
    changed = (cache.k != before).any(-1).any(-1).nonzero().cpu().numpy().tolist()
    assert changed == [[int(table[0, 0]), 3]]
    out = {n: torch.full((5, 1, 64), 7.0, device="cuda") for n in ("k", "v")}
    fb.cache_read(cache, seq, pos, out=out)
    assert bool((out["k"][1:] == 7.0).all()) and bool((out["k"][0] == 1.0).all())
    assert fb.STATUS[fb.fa_back_get_error()] == "FA_ERR_PAGE"
    # decode: keys on an invalid page are masked
    fb.cache_append(x[:1].expand(16, 1, 64), x[:1].expand(16, 1, 64), cache, cuda(np.ones(16, np.int32)), cuda(np.arange(16, dtype=np.int32)))
    got = fb.paged_decode(torch.ones(2, 1, 64, device="cuda"), cache, cuda(np.array([0, 20], np.int32)), scale=0.1)
    torch.cuda.synchronize()
    assert fb.STATUS[fb.fa_back_get_error()] == "FA_ERR_PAGE"
    assert bool((got["O"][1] == 1.0).all()) and abs(float(got["lse"][1, 0]) - (6.4 + np.log(16))) < 1e-5
    # a length beyond the table counts as the whole table
    got = fb.paged_decode(torch.ones(2, 1, 64, device="cuda"), cache, cuda(np.array([-1, 2000000000], np.int32)), scale=0.1)
    assert bool((got["O"][1] == 1.0).all())
    assert fb.STATUS[fb.fa_back_get_error()] == "FA_ERR_PAGE"


# ------------------------------------------------------------------------------------------------
# single-token attention

def check_decode(fb, p, H, act="f32", softcap=0.0, alibi=False, sinks=False, seed=0, q_amp=1.0, scale=None):
    rng = np.random.default_rng(seed)
    B = len(p.lens)
    q = torch.from_numpy((q_amp * rng.standard_normal((B, H, p.D))).astype(np.float32)).to(DT[act]).cuda()
    scale = p.D ** -0.5 if scale is None else scale
    sl = (2.0 ** (-8.0 * (np.arange(H) + 1) / H)).astype(np.float32) if alibi else None
    sk = (1.0 + rng.standard_normal(H)).astype(np.float32) if sinks else None
    cache = p.on_gpu(fb, torch)
    out = {"O": torch.full((B, H, p.Dv), 7.0, dtype=DT[act], device="cuda"), "lse": torch.full((B, H), 7.0, device="cuda")}
    fb.paged_decode(q, cache, cuda(np.array(p.lens, np.int32)), scale=scale, alibi_slopes=cuda(sl), softcap=softcap, sinks=cuda(sk), out=out)
    torch.cuda.synchronize()
    assert fb.fa_back_get_error() == 0
    O, lse, mag, smag = R.decode(p, q.float().cpu().numpy(), scale, softcap, sl, sk)
    tol_O, tol_lse = R.decode_tolerance(p, mag, smag, act)
    live = np.array(p.lens) >= 0
    got_O, got_lse = out["O"].float().cpu().numpy(), out["lse"].cpu().numpy()
    assert np.all(got_O[~live] == 7.0) and np.all(got_lse[~live] == 7.0)  # padding slots
    within(got_lse[live], lse[live], tol_lse[live], "lse")
    within(got_O[live], O[live], (tol_O + half_step(act, O))[live], "O")
    return q, cache, out


LENS = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 129, 300, 1000, -1, 511]


@pytest.mark.parametrize("kt", [F32, F16, Q8, Q4])
@pytest.mark.parametrize("vt", [F32, F16, Q8, Q4])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_decode_types(fb, kt, vt, D):
    p = R.Paged(kt * 16 + vt * 4 + D, LENS, 2, D, D, kt, vt, 16)
    check_decode(fb, p, 6, seed=D)


SHAPES = {  # lens, H, Hkv, D, Dv, kt, vt, act, page, opts
    "mha": ([100, 7, 0], 3, 3, 64, 64, Q8, Q8, "f32", 16, {}),
    "mqa_20": ([1300, 1, 40], 20, 1, 128, 128, Q8, Q4, "f32", 64, {}),
    "group_8": ([777], 16, 2, 256, 256, F16, F16, "bf16", 32, {}),
    "group_9": ([600, 601], 18, 2, 64, 64, Q4, F16, "f16", 48, {}),
    "group_16_d256": ([2000, 3], 16, 1, 256, 256, Q8, Q8, "bf16", 64, {}),
    "dv_smaller": ([500, 33], 12, 2, 256, 64, Q8, F16, "f32", 16, {}),
    "dv_larger": ([500, 33], 4, 2, 64, 256, F16, Q8, "f32", 16, {}),
    "page_1": ([70, 17], 4, 2, 64, 64, F16, F32, "f32", 1, {}),
    "page_3": ([200, 16], 4, 4, 128, 128, Q8, Q8, "f32", 3 * 2, {}),
    "page_5": ([250, 5], 4, 2, 64, 64, Q8, Q4, "f32", 20, {}),
    "page_40": ([900, 39, 40, 41], 6, 1, 256, 256, Q4, Q8, "f32", 40, {}),
    "page_4096": ([5000, 100], 6, 1, 128, 128, Q8, Q8, "f32", 4096, {}),
    "softcap": ([333, 2], 8, 2, 128, 128, Q8, Q8, "f32", 16, dict(softcap=2.0, q_amp=3.0)),
    "alibi": ([333, 2, 0], 8, 2, 128, 128, F16, Q8, "f32", 16, dict(alibi=True)),
    "sinks": ([333, 1, 0], 8, 2, 128, 128, Q8, F16, "f32", 16, dict(sinks=True)),
    "all_ext": ([800, 1, 0, 64], 12, 2, 256, 256, Q4, Q8, "f16", 40, dict(softcap=30.0, alibi=True, sinks=True)),
    "sharp": ([1500, 64], 6, 2, 64, 64, Q8, Q8, "f32", 64, dict(q_amp=30.0)),
    "small_q": ([1500, 64], 6, 2, 64, 64, Q8, Q8, "f32", 64, dict(q_amp=1e-18, scale=1e17)),
    "large_q": ([1500, 64], 6, 2, 64, 64, F16, F32, "f32", 64, dict(q_amp=1e18, scale=1e-19)),
    "many_sequences": (list(range(0, 300)), 4, 1, 64, 64, Q8, Q8, "bf16", 16, {}),
    "long_one": ([40000], 8, 2, 128, 128, Q8, Q8, "f32", 64, {}),
    "large_batch_one_long": ([9000] + [0, 1, 17, 40] * 75, 6, 2, 64, 64, Q8, Q8, "f32", 16, {}),
    "large_batch_split": ([700] * 260, 8, 8, 64, 64, F16, Q4, "bf16", 40, {}),
    "fits_less_than_a_chunk": ([3000, 2900] + [10] * 60, 16, 8, 64, 64, Q8, F16, "bf16", 8, {}),
    "hkv_3_page_8": ([333, 8, 9, 1000], 6, 3, 128, 128, Q8, Q8, "f32", 8 * 3, {}),
    "long_and_short": ([20011, 1, 3, 0, 9001, 17] + [5] * 30, 12, 2, 128, 128, Q8, Q4, "f32", 64, {}),
}


@pytest.mark.parametrize("name", sorted(SHAPES))
def test_decode_shapes(fb, name):
    lens, H, Hkv, D, Dv, kt, vt, act, page, opts = SHAPES[name]
    p = R.Paged(sorted(SHAPES).index(name) + 900, lens, Hkv, D, Dv, kt, vt, page)
    check_decode(fb, p, H, act, seed=1, **opts)


@pytest.mark.parametrize("seed", range(24))
def test_decode_random(fb, seed):
    """Seeded random shapes, types, pages, lengths and score extensions."""
    r = np.random.default_rng(4000 + seed)
    pick = lambda *a: a[int(r.integers(len(a)))]  # noqa: E731
    D, Dv = pick(64, 128, 256), pick(64, 128, 256)
    kt, vt = pick(F32, F16, Q8, Q4), pick(F32, F16, Q8, Q4)
    Hkv, G, B = pick(1, 2, 3, 4, 5), pick(1, 2, 3, 5, 8, 9, 13), int(r.integers(1, 12))
    page = pick(8, 16, 24, 32, 40, 48, 64, 100, 256)
    if page * Hkv * synth.row_bytes(kt, D) % 16 or page * Hkv * synth.row_bytes(vt, Dv) % 16:
        page = 16
    lens = [int(x) for x in np.exp(r.uniform(-0.5, np.log(3000), B))]
    p = R.Paged(seed, lens, Hkv, D, Dv, kt, vt, page)
    check_decode(fb, p, G * Hkv, pick("f32", "f16", "bf16"), softcap=pick(0.0, 0.0, 20.0), alibi=pick(True, False),
                 sinks=pick(True, False), seed=seed)


@pytest.mark.parametrize("amp", [1e-4, 1e4])
@pytest.mark.parametrize("vt", [F32, F16, Q8, Q4])
def test_decode_value_range(fb, vt, amp):
    """Values far from one: block scales and products leave neither end of the working types' range."""
    p = R.Paged(vt + 40, [500, 30], 2, 128, 128, Q8, vt, 16, v_amp=amp)
    check_decode(fb, p, 8)


@pytest.mark.parametrize("page", [16, 64, 40, 20])
@pytest.mark.parametrize("kt, vt", [(Q8, Q8), (F16, F16)])
def test_decode_around_invalid_pages(fb, kt, vt, page):
    """Pages without a valid number in the middle of long sequences: their keys are masked, those behind them count."""
    p = R.Paged(page + kt, [4000, 700, 33], 2, 128, 128, kt, vt, page)
    rng = np.random.default_rng(page)
    bad = rng.random(p.table.shape) < 0.2
    bad[:, 0] = [False, True, False]
    p.table[bad] = np.where(rng.random(bad.sum()) < 0.5, -1, 10 ** 6)
    q, qa = act_array(rng, (3, 8, 128), "f32")
    got = fb.paged_decode(q, p.on_gpu(fb, torch), cuda(np.array(p.lens, np.int32)), scale=0.1)
    torch.cuda.synchronize()
    assert fb.STATUS[fb.fa_back_get_error()] == "FA_ERR_PAGE"
    for b, n in enumerate(p.lens):
        keep = ~bad[b, np.arange(n) // page]
        p.kd[b], p.vd[b], p.lens[b] = p.kd[b][keep], p.vd[b][keep], int(keep.sum())
    O, lse, mag, smag = R.decode(p, qa, 0.1)
    tol_O, tol_lse = R.decode_tolerance(p, mag, smag, "f32")
    within(got["O"].cpu().numpy(), O, tol_O, "O")
    within(got["lse"].cpu().numpy(), lse, tol_lse, "lse")


@pytest.mark.parametrize("pair", [(16, 64), (40, 20)])
def test_decode_calls_that_overlap(fb, pair):
    """Calls on two streams at once, each with a workspace of its own."""
    ps = [R.Paged(90 + i, [6000, 50, 900], 2, 128, 128, Q8, Q8, page) for i, page in enumerate(pair)]
    want = [check_decode(fb, p, 8, seed=i) for i, p in enumerate(ps)]
    lens = [cuda(np.array(p.lens, np.int32)) for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for (q, cache, _), n, s in zip(want, lens, streams):
            got.append(fb.paged_decode(q, cache, n, scale=128 ** -0.5, stream=s))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        out = want[i % 2][2]
        assert torch.equal(g["O"], out["O"]) and torch.equal(g["lse"], out["lse"])


@pytest.mark.parametrize("kt", [F32, F16, Q8, Q4])
@pytest.mark.parametrize("q_amp, k_amp, scale", [(1e-39, 1.0, 1.0), (1e-36, 1.0, 1e36), (1e37, 1.0, 1e-37), (1e-30, 1e3, 1e27)])
def test_decode_query_range(fb, kt, q_amp, k_amp, scale):
    """Queries near both ends of f32's range (denormal ones too), with keys and a scale that bring the scores back."""
    p = R.Paged(60 + kt, [900, 30], 2, 128, 128, kt, Q8, 16, k_amp=k_amp)
    check_decode(fb, p, 8, q_amp=q_amp, scale=scale / 11.3)


def test_decode_f32_keys_beyond_other_types(fb):
    """f32 keys of 1e30: the products are those of q and k themselves."""
    p = R.Paged(71, [900, 30], 2, 64, 64, F32, F32, 16, k_amp=1e30)
    check_decode(fb, p, 4, q_amp=1e-30)


@pytest.mark.parametrize("sinks", [False, True])
def test_decode_nan_stays_with_its_head(fb, sinks):
    p = R.Paged(72, [30, 2500, 0], 2, 64, 64, Q8, F16, 16)
    q, qa = act_array(np.random.default_rng(3), (3, 6, 64), "f32")
    sk = np.zeros(6, np.float32) if sinks else None
    O, lse, mag, smag = R.decode(p, qa, 0.125, sinks=sk)
    tol_O, tol_lse = R.decode_tolerance(p, mag, smag, "f32")
    q[:, 4, 7] = float("nan")
    got = fb.paged_decode(q, p.on_gpu(fb, torch), cuda(np.array(p.lens, np.int32)), scale=0.125, sinks=cuda(sk))
    gO, gl = got["O"].cpu().numpy(), got["lse"].cpu().numpy()
    assert np.isnan(gO[:2, 4]).all() and np.isnan(gl[:2, 4]).all()
    rest = [0, 1, 2, 3, 5]
    within(gO[:, rest], O[:, rest], tol_O[:, rest], "O")
    within(gl[:, rest], lse[:, rest], tol_lse[:, rest], "lse")
    assert not gO[2].any() and np.array_equal(gl[2], lse[2])


def test_decode_equal_calls_and_streams(fb):
    p = R.Paged(5, [3000, 10, 700], 2, 128, 128, Q8, Q8, 16)
    q, cache, out = check_decode(fb, p, 8)
    lens = cuda(np.array(p.lens, np.int32))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a = fb.paged_decode(q, cache, lens, scale=128 ** -0.5)
    b = fb.paged_decode(q, cache, lens, scale=128 ** -0.5, stream=s)
    torch.cuda.synchronize()
    for x in (a, b):
        assert torch.equal(x["O"], out["O"]) and torch.equal(x["lse"], out["lse"])
    # a query inside a fused projection, rows off 16 bytes
    fused = torch.zeros(3 * 12 * 128 + 1, device="cuda")[1:].view(3, 12, 128)
    fused[:, 1:9] = q
    c = fb.paged_decode(fused[:, 1:9], cache, lens, scale=128 ** -0.5)
    assert torch.equal(c["O"], out["O"])


def test_decode_gives_up_on_a_wait(fb):
    """With a wait limit of zero the kernel records a timeout, drains its copies and returns; the next call
    is right again."""
    p = R.Paged(8, [3000, 500, 1000], 2, 256, 256, Q8, Q8, 64)
    q, cache, out = check_decode(fb, p, 8)
    assert fb.fa_back_test_wait_limit(0) == 0
    fb.paged_decode(q, cache, cuda(np.array(p.lens, np.int32)), scale=256 ** -0.5)
    assert fb.STATUS[fb.fa_back_get_error()] == "FA_ERR_TIMEOUT"
    again = fb.paged_decode(q, cache, cuda(np.array(p.lens, np.int32)), scale=256 ** -0.5)
    assert torch.equal(again["O"], out["O"]) and fb.fa_back_get_error() == 0


def test_decode_in_a_graph_follows_lengths_and_rows(fb):
    """A captured append + decode step: replays take the lengths, positions and rows of the moment."""
    p = R.Paged(6, [90, 300], 2, 64, 64, Q8, Q8, 16)
    H, D = 4, 64
    cache = p.on_gpu(fb, torch)
    wide = torch.cat([cache.page_table, torch.tensor([[200, 201, 202], [203, 204, 205]], dtype=torch.int32, device="cuda")], 1)
    grow = [torch.zeros((206 - x.shape[0], *x.shape[1:]), dtype=torch.uint8, device="cuda") for x in (cache.k, cache.v)]
    cache = fb.PagedCache(torch.cat([cache.k, grow[0]]), Q8, torch.cat([cache.v, grow[1]]), Q8, wide.contiguous(), D=D, Dv=D)
    lens = cuda(np.array(p.lens, np.int32))
    seq = torch.arange(2, dtype=torch.int32, device="cuda")
    q, k, v = (torch.randn(2, h, D, device="cuda") for h in (H, 2, 2))
    ws = fb.Workspace("cuda")
    rope = fb.rope_frequencies(D)

    def step():
        pos = lens.clone()
        fb.cache_append(k, v, cache, seq, pos, rope=rope)
        lens.add_(1)
        return fb.paged_decode(q, cache, lens, scale=D ** -0.5, workspace=ws)

    ws.get(cache.decode_workspace_size(H))
    start = cache.k.clone(), cache.v.clone(), lens.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    cache.k.copy_(start[0]), cache.v.copy_(start[1]), lens.copy_(start[2])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    inputs = [[torch.randn_like(x) for x in (q, k, v)] for _ in range(20)]
    outs = []
    for a in inputs:
        q.copy_(a[0]), k.copy_(a[1]), v.copy_(a[2])
        g.replay()
        outs.append(got["O"].clone())
    final = cache.k.clone()
    cache.k.copy_(start[0]), cache.v.copy_(start[1]), lens.copy_(start[2])
    for a, o in zip(inputs, outs):
        q.copy_(a[0]), k.copy_(a[1]), v.copy_(a[2])
        assert torch.equal(step()["O"], o)
    assert torch.equal(cache.k, final) and lens.tolist() == [110, 320]
    assert fb.fa_back_get_error() == 0


def test_decode_beyond_two_gigabytes(fb):
    """Pages whose byte offsets need more than 32 bits."""
    Hkv, D, page, n_pages = 4, 256, 64, 10000  # 2.6 GB of f32 keys, 1.3 GB of f16 values
    k = torch.empty((n_pages, page, Hkv, 4 * D), dtype=torch.uint8, device="cuda")
    v = torch.empty((n_pages, page, Hkv, 2 * D), dtype=torch.uint8, device="cuda")
    small = R.Paged(77, [150, 64], Hkv, D, D, F32, F16, page)
    far = np.array([[9999, 0, 9400], [8800, 9998, 5000]], np.int32)
    for b in range(2):
        for i in range(small.max_pages):
            k[int(far[b, i])] = torch.from_numpy(small.k[small.table[b, i]]).cuda()
            v[int(far[b, i])] = torch.from_numpy(small.v[small.table[b, i]]).cuda()
    rng = np.random.default_rng(1)
    q, qa = act_array(rng, (2, 8, D), "f32")
    cache = fb.PagedCache(k, F32, v, F16, cuda(far), D=D, Dv=D)
    got = fb.paged_decode(q, cache, cuda(np.array([150, 64], np.int32)), scale=D ** -0.5)
    O, lse, mag, smag = R.decode(small, qa, D ** -0.5)
    tol_O, tol_lse = R.decode_tolerance(small, mag, smag, "f32")
    within(got["O"].cpu().numpy(), O, tol_O, "O")
    within(got["lse"].cpu().numpy(), lse, tol_lse, "lse")
    x, xa = act_array(rng, (2, Hkv, D), "f32")
    seq, pos = cuda(np.array([0, 1], np.int32)), cuda(np.array([150, 64], np.int32))
    fb.cache_append(x, x, cache, seq, pos)
    back = fb.cache_read(cache, seq, pos)
    assert torch.equal(back["k"], x) and torch.equal(back["v"], x.half().float())
    assert fb.fa_back_get_error() == 0


def test_both_forms_of_the_wrappers_agree(fb, monkeypatch):
    """The calls with and without the marshalling module: the same results, keys and types."""
    from flash_attention_backward_gb300 import paged
    assert paged._fast is not None
    rng = np.random.default_rng(31)
    p = R.Paged(31, [70, 0, 200], 2, 128, 64, Q8, F16, 16)
    cache = p.on_gpu(fb, torch)
    (q, _), (k, _), (v, _) = (act_array(rng, (3, h, d), "bf16") for h, d in ((6, 128), (2, 128), (2, 64)))
    w, rope = torch.rand(128, device="cuda") + 0.5, fb.rope_frequencies(128)
    seq, pos = cuda(np.array([0, 2, 2], np.int32)), cuda(np.array([5, 17, 180], np.int32))
    lens = cuda(np.array(p.lens, np.int32))
    calls = [
        lambda: fb.paged_decode(q, cache, lens, scale=0.1, softcap=20.0, sinks=w[:6].contiguous()),
        lambda: fb.cache_read(cache, seq, pos, dtype=torch.bfloat16),
        lambda: fb.qk_norm_rope(q, k, pos, wq=w, wk=w, rope=rope, rope_style=fb.FA_ROPE_PAIRS, dtype=torch.float32),
        lambda: fb.qk_norm_rope(q, None, None, wq=w),
        lambda: fb.qk_norm_rope_backward(q, k, q, k, pos, wq=w, wk=w, rope=rope),
        lambda: fb.qk_norm_rope_backward(q.float(), None, q, None, pos, rope=rope),
    ]
    was = paged._fast
    for name in ("norm", "norm_back", "append", "read", "decode"):
        assert callable(getattr(was, name))
    fast = [c() for c in calls]
    fb.cache_append(k, v, cache, seq, pos, k_norm=w, rope=rope)
    after = cache.k.clone(), cache.v.clone()
    cache.k.copy_(torch.from_numpy(p.k)), cache.v.copy_(torch.from_numpy(p.v))
    monkeypatch.setattr(paged, "_fast", None)
    monkeypatch.setattr(paged, "_plain", False)
    for c, f in zip(calls, fast):
        g = c()
        assert list(g) == list(f)
        for n in g:
            assert (g[n] is None) == (f[n] is None)
            assert g[n] is None or (g[n].dtype == f[n].dtype and torch.equal(g[n], f[n])), n
    fb.cache_append(k, v, cache, seq, pos, k_norm=w, rope=rope)
    assert torch.equal(cache.k, after[0]) and torch.equal(cache.v, after[1])


# ------------------------------------------------------------------------------------------------
# together with the attention of fa_back.h

def test_a_layer_end_to_end(fb):
    """norm + rotation -> paged append -> single-token attention, against forward() over the same cache read
    back raw; then backward() on it and the gradient through the rotation and the norm."""
    rng = np.random.default_rng(21)
    T, H, Hkv, D, page = 200, 8, 2, 128, 16
    (xq, qa), (xk, ka), (xv, _) = (act_array(rng, (T, h, D), "f32") for h in (H, Hkv, Hkv))
    wq, wk = (torch.rand(D, device="cuda") + 0.5 for _ in range(2))
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    seq = torch.zeros(T, dtype=torch.int32, device="cuda")
    rope = fb.rope_frequencies(D)
    y = fb.qk_norm_rope(xq, xk, pos, wq=wq, wk=wk, rope=rope)
    cache, _ = empty_cache(fb, 1, 13, page, Hkv, D, D, Q8, Q8)
    fb.cache_append(xk, xv, cache, seq, pos, k_norm=wk, rope=rope)
    other, _ = empty_cache(fb, 1, 13, page, Hkv, D, D, Q8, Q8)
    fb.cache_append(y["k"], xv, other, seq, pos)  # the same keys, normalised and rotated beforehand
    assert torch.equal(cache.k, other.k) and torch.equal(cache.v, other.v)
    raw = fb.cache_read(cache, seq, pos, dtype=torch.uint8)
    kw = dict(H=H, Hkv=Hkv, D=D, Dv=D, M=T, scale=D ** -0.5, causal=True)
    f = fb.forward(y["q"], raw["k"], Q8, raw["v"], Q8, **kw)
    last = fb.paged_decode(y["q"][-1:], cache, torch.tensor([T], dtype=torch.int32, device="cuda"), scale=D ** -0.5)
    # forward() rounds its operands to binary16; its own tests hold it to NMSE 1e-5
    d = (last["O"][0] - f["O"][-1]).double()
    assert float((d * d).sum() / (f["O"][-1].double() ** 2).sum()) <= 1e-5
    assert float((last["lse"][0] - f["lse"][-1]).abs().max()) < 1e-3
    dO = torch.randn(T, H, D, device="cuda")
    b = fb.backward(y["q"], raw["k"], Q8, raw["v"], Q8, dO, **kw)
    g = fb.qk_norm_rope_backward(b["dQ"], b["dK"], xq, xk, pos, wq=wq, wk=wk, rope=rope)
    for n, x, w, gy in (("q", qa, wq, b["dQ"]), ("k", ka, wk, b["dK"])):
        dx, dw, *_ = back_reference(x, w.cpu().numpy(), gy.cpu().numpy(), pos.cpu().numpy(), D, True)
        for got, ref in ((g["d" + n], dx), (g["dw" + n], dw)):
            e = got.double().cpu().numpy() - ref
            assert (e ** 2).sum() <= (1e-5 ** 2) * (ref ** 2).sum()
    assert fb.fa_back_get_error() == 0
