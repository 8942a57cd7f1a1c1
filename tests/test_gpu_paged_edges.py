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


ROTATIONS = [(64, 0, True), (64, 0, False), (64, 16, True), (64, 64, True), (128, 32, True), (128, 34, False), (128, 128, False),
             (256, 96, True), (256, 2, False), (256, 256, True)]


def not_finite(N, H, D, seed):
    """Ordinary heads with one infinity or NaN each, every component in turn."""
    x = np.random.default_rng(seed).standard_normal((N, H, D)).astype(np.float32)
    n = np.arange(N * H)
    x.reshape(N * H, D)[n, n % D] = np.array([np.inf, np.nan, -np.inf], np.float32)[n // D % 3]
    return x


def turned(x, pos, n_rot, halves, sign=1.0):
    """The definition: (a cos - b sin, a sin + b cos) for the pairs, nothing for the rest."""
    y = x.astype(np.float64)
    if n_rot:
        with np.errstate(invalid="ignore"):
            y = R.rotate(y, pos, n_rot, 10000.0, halves, sign)
    return y


def same_kinds(got, ref, tol, what):
    assert np.array_equal(np.isnan(got), np.isnan(ref)), (what, int(np.isnan(got).sum()), int(np.isnan(ref).sum()))
    inf = np.isinf(ref)
    assert np.array_equal(got[inf], ref[inf]) and np.array_equal(np.isinf(got), inf), what
    fin = np.isfinite(ref)
    assert np.abs(got[fin] - ref[fin]).max() <= tol, what


@pytest.mark.parametrize("D, n_rot, halves", ROTATIONS)
def test_a_value_that_is_not_finite_touches_its_pair_alone(fb, D, n_rot, halves):
    """Rotation without a norm, its gradient and an append to F32 and F16 rows: an infinity or a NaN enters the two
    components of its pair, as in the definition, and an unrotated one is kept as it is."""
    H, Hkv = 6, 2
    N = 3 * D // Hkv  # every component with every kind, in the keys too
    q, k = not_finite(N, H, D, D), not_finite(N, Hkv, D, D + 1)
    # positions whose angles are off the axes: cos and sin are not 0 (inf * 0)
    pos = np.random.default_rng(n_rot).integers(1, 5000, N).astype(np.int32)
    rope = fb.rope_frequencies(n_rot, 10000.0) if n_rot else None
    kw = dict(rope=rope, rope_style=int(halves))
    tol = 20 * U * 12  # 20 u of the pair's magnitude, which is below 12 for these normals
    got = fb.qk_norm_rope(cuda(q), cuda(k), cuda(pos), **kw)
    back = fb.qk_norm_rope_backward(cuda(q), cuda(k), cuda(q), cuda(k), cuda(pos), **kw)
    for n, x in (("q", q), ("k", k)):
        same_kinds(got[n].cpu().numpy().astype(np.float64), turned(x, pos, n_rot, halves), tol, n)
        same_kinds(back["d" + n].cpu().numpy().astype(np.float64), turned(x, pos, n_rot, halves, -1.0), tol, "d" + n)
    for ty in (F32, F16):
        cache, _ = empty_cache(fb, 1, -(-5000 // 64), 64, Hkv, D, D, ty, ty)
        at = np.random.default_rng(1).permutation(np.arange(1, 5000))[:N].astype(np.int32)
        seq = cuda(np.zeros(N, np.int32))
        fb.cache_append(cuda(k), cuda(k), cache, seq, cuda(at), **kw)
        rows = fb.cache_read(cache, seq, cuda(at))
        half = 0.0 if ty == F32 else 2.0 ** -11 * 12
        same_kinds(rows["k"].cpu().numpy().astype(np.float64), turned(k, at, n_rot, halves), tol + half, "rows k")
        same_kinds(rows["v"].cpu().numpy().astype(np.float64), k.astype(np.float64), half, "rows v")
    assert fb.fa_back_get_error() == 0


@pytest.mark.parametrize("N, H, Hkv, D, act", [(3000, 6, 2, 128, "bf16"), (500, 3, 1, 256, "f32"), (2, 1, 1, 64, "f32")])
def test_gradient_gives_up_on_a_wait(fb, N, H, Hkv, D, act):
    """With a wait limit of zero the gradient's kernel records a timeout, drains its copies and returns; the next
    call is right again, bit for bit."""
    rng = np.random.default_rng(N)
    (q, _), (k, _), (gq, _), (gk, _) = (act_array(rng, (N, h, D), act) for h in (H, Hkv, H, Hkv))
    w, pos = torch.rand(D, device="cuda") + 0.5, torch.arange(N, dtype=torch.int32, device="cuda")
    kw = dict(wq=w, wk=w, rope=fb.rope_frequencies(D))
    want = fb.qk_norm_rope_backward(gq, gk, q, k, pos, **kw)
    assert fb.fa_back_get_error() == 0
    assert fb.fa_back_test_wait_limit(0) == 0
    fb.qk_norm_rope_backward(gq, gk, q, k, pos, **kw)
    assert fb.STATUS[fb.fa_back_get_error()] == "FA_ERR_TIMEOUT"
    again = fb.qk_norm_rope_backward(gq, gk, q, k, pos, **kw)
    assert fb.fa_back_get_error() == 0
    for n in want:
        assert torch.equal(again[n], want[n]), n


def test_rotation_angles_to_32_bits(fb):
    """cos and sin themselves (the rotation of (1, 0)), at any frequency and position: within 1.5 units of the result
    (one of sincospi's, half of the rounding behind it; a unit is at most 2^-23 of the value) and the 1.5e-9 rad
    that an angle of 32 bits is off.  Both ways, and on the way into a cache."""
    rng = np.random.default_rng(41)
    N, D = 4000, 64
    freq = rng.integers(-2 ** 63, 2 ** 63, 32)
    rope = cuda(freq)
    x = np.zeros((N, 1, D), np.float32)
    for halves in (True, False):
        first, second = (np.arange(32), np.arange(32) + 32) if halves else (2 * np.arange(32), 2 * np.arange(32) + 1)
        x[:] = 0.0
        x[:, 0, first] = 1.0

        def check(got, pos, sign, what):
            turns = np.array([[(int(p) * int(f)) % 2 ** 64 for f in freq] for p in pos], dtype=object)
            t = (turns / 2 ** 64).astype(np.float64)  # (2^-53 turns: nothing here)
            for at, ref in ((first, np.cos(2 * np.pi * t)), (second, sign * np.sin(2 * np.pi * t))):
                off = np.abs(got[:, 0, at] - ref)
                assert (off <= 1.5 * 2.0 ** -23 * np.abs(ref) + 1.5e-9).all(), (what, off.max())

        pos = rng.integers(-2 ** 31, 2 ** 31, N).astype(np.int32)
        kw = dict(rope=rope, rope_style=int(halves))
        check(fb.qk_norm_rope(cuda(x), None, cuda(pos), **kw)["q"].double().cpu().numpy(), pos, 1.0, "forward")
        check(fb.qk_norm_rope_backward(cuda(x), None, cuda(x), None, cuda(pos), **kw)["dq"].double().cpu().numpy(), pos, -1.0, "back")
        cache, _ = empty_cache(fb, 1, -(-N // 64), 64, 1, D, D, F32, F32)
        at, seq = np.arange(N, dtype=np.int32), cuda(np.zeros(N, np.int32))
        fb.cache_append(cuda(x), cuda(x), cache, seq, cuda(at), **kw)
        check(fb.cache_read(cache, seq, cuda(at))["k"].double().cpu().numpy(), at, 1.0, "append")


@pytest.mark.parametrize("vt", [Q8, Q4])
def test_weights_of_quantised_values_keep_their_bits(fb, vt):
    """Two keys, of which one has values: O is that key's weight, 1 / (1 + exp(-a)), times whole numbers.

    Per output, in u = 2^-24 of it: the score a is exact (11 bits, a key of one 1), its product with log2 e two
    roundings, 1.5 a <= 1.5; either exponential 4 (2^-22), which enter by 1 - weight < 0.74: 6; the parts of
    the weight are exact, their three products are summed with up to 2 lost each: 6; the sum of weights, the
    factors of the join, the division and its product: 6.  Together under 24.  (Two bf16 parts alone: up to 128.)"""
    B, H, D = 64, 8, 64
    rng = np.random.default_rng(51)
    p = R.Paged(51, [2] * B, 1, D, D, F16, vt, 16)
    a = rng.integers(1, 1024, (B, H)) / 1024.0 * rng.choice([-1.0, 1.0], (B, H))
    q = np.zeros((B, H, D), np.float32)
    q[..., 0] = a
    k, v = np.zeros((B, 2, D), np.float16), np.zeros((B, 2, 1, D), np.float32)
    k[:, 0, 0] = 1.0
    v[:, 0, 0] = rng.integers(-126, 127, (B, D)) if vt == Q8 else rng.integers(-7, 8, (B, D))
    v[:, 0, 0, ::32] = 127 if vt == Q8 else -8  # the block scale is 1
    p.k[p.table[:, 0], :2, 0] = k.view(np.uint8)
    p.v[p.table[:, 0], :2] = R.synth.quantize_rows(v, vt)
    got = fb.paged_decode(cuda(q), p.on_gpu(fb, torch), cuda(np.array(p.lens, np.int32)), scale=1.0)
    ref = (1.0 / (1.0 + np.exp(-a)))[..., None] * v[:, 0].astype(np.float64)
    off = np.abs(got["O"].double().cpu().numpy() - ref)
    assert (off <= 24 * U * np.abs(ref)).all(), (off / np.maximum(np.abs(ref), 1e-30)).max() / U
    assert fb.fa_back_get_error() == 0


@pytest.mark.parametrize("ty", [F32, F16, Q8, Q4])
def test_f32_outputs_of_long_sequences(fb, ty):
    """A batch that fills the card with whole sequences: each warp sums 188 tiles of 16 keys.

    The 2-norm of the error over that of O, in u = 2^-24.  O is a sum of terms of random sign, so what is off
    by d in each term is off by d in O: score (22 bits of q, 4 rounded steps), exponential and parts of a weight,
    each at random, below 6 in the root mean square; products and sum of a tile, cut off up to 3 times, 6 of a sum
    that is 1 / sqrt(750) of the whole: nothing; 188 rounded additions of at most 1 at random, whose sizes grow to
    the final one's: sqrt(188 / 3 / 2) = 6; the sum of weights 188 of one sign, at random: sqrt(188 / 3) = 8.
    Together 12; 32 are allowed.  (In one chain through the tensor core, two or six cuts a tile of one unit on
    average, all towards zero: 75 to 375.)"""
    B, L, H, D, page = 80, 12000, 64, 64, 64
    gen = torch.Generator(device="cuda").manual_seed(61 + ty)
    table = torch.arange(B * 188, dtype=torch.int32, device="cuda").view(B, 188)
    pools = [torch.zeros(B * 188, page, 1, R.synth.row_bytes(ty, D), dtype=torch.uint8, device="cuda") for _ in range(2)]
    cache = fb.PagedCache(pools[0], ty, pools[1], ty, table, D=D, Dv=D)
    q = torch.randn(B, H, D, generator=gen, device="cuda")
    pos, ref = torch.arange(L, dtype=torch.int32, device="cuda"), torch.empty(B, H, D, dtype=torch.float64, device="cuda")
    for b in range(B):
        x = torch.randn(2, L, 1, D, generator=gen, device="cuda")
        fb.cache_append(x[0], x[1], cache, torch.full_like(pos, b), pos)
        raw = fb.cache_read(cache, torch.full_like(pos, b), pos, dtype=torch.uint8)
        k, v = (cuda(R.oracle.dequant(raw[n][:, 0].cpu().numpy(), ty, D).reshape(L, D)).double() for n in ("k", "v"))
        ref[b] = torch.softmax(q[b].double() @ k.T * D ** -0.5, -1) @ v
    got = fb.paged_decode(q, cache, torch.full((B,), L, dtype=torch.int32, device="cuda"), scale=D ** -0.5)
    off = float((got["O"].double() - ref).norm() / ref.norm())
    assert off <= 32 * U, off / U
    assert fb.fa_back_get_error() == 0


def test_f32_values_are_rounded_to_their_parts(fb):
    """One key: O is its f32 value p v / p, with v and the weight p (2^7 but for the rounding of its exponent) each in
    parts of 11 and 11 bits.  In u: rounded, v and p are off by at most 4 (two of 13 lower bits go; a granule is 2) and
    on average by nothing; the product of the second parts, 2^-12 of 2^-12, is left out: 1; the sum of the three
    products is cut twice, the first time beside a sum of 2^-11 (nothing), the second by less than 2, 0.7 on average
    over a binade; division and its product 2.  Together 13 at most, and in the mean of 512 weights and 131072 values
    0.7 (+ 0.1 left out) with a deviation of 1 / sqrt(512) + 4 / sqrt(131072) = 0.06: under 1.2.  (Parts that are cut
    off: 1.3 more in the mean for v, 1.3 for p.)"""
    B, Hkv, D = 64, 8, 256
    p = R.Paged(71, [1] * B, Hkv, 64, D, F16, F32, 16)
    q, _ = act_array(np.random.default_rng(71), (B, Hkv, 64), "f32")
    got = fb.paged_decode(q, p.on_gpu(fb, torch), cuda(np.ones(B, np.int32)), scale=0.1)
    v = np.stack([x[0] for x in p.vd])
    rel = (got["O"].double().cpu().numpy() - v) / np.abs(v) * np.sign(v) / U
    assert np.abs(rel).max() <= 13.0, np.abs(rel).max()
    assert abs(rel.mean()) <= 1.2, rel.mean()


@pytest.mark.parametrize("off", [0, 1])
def test_weights_gradient_over_many_rows(fb, off):
    """dw of 4 million rows of one head, 1724 a lane, from aligned rows and from rows off 16 bytes; the 2-norm of the error
    over that of dw, in u = 2^-24.  Terms have random signs: an error d of each is one of d in the sum: two rounded
    products and r, 1.2 in the root mean square.  A sum of n terms: each addition rounds by 0.3 (a half at most, evenly)
    of a unit of the sum so far, of up to 2: 0.3 sqrt(n / 2) of the last one; 41 terms and 42 of those sums: 1.4 and
    1.4; the rest keeps what its roundings lose, but for the last two, 0.4.  Together 2.4, and 3.2 are allowed (all in one f32 sum: 8.8)."""
    N, D = 4193000, 64
    gen = torch.Generator(device="cuda").manual_seed(81)
    x, gy = (torch.randn(N * D + 8, generator=gen, device="cuda").bfloat16() for _ in range(2))
    x, gy = x[off:off + N * D].view(N, 1, D), gy[:N * D].view(N, 1, D)
    w = torch.rand(D, generator=gen, device="cuda") + 0.5
    got = fb.qk_norm_rope_backward(gy, None, x, None, None, wq=w)["dwq"].double()
    ref = torch.zeros(D, dtype=torch.float64, device="cuda")
    for a, g in zip(x.split(1 << 19), gy.split(1 << 19)):
        a = a.double()
        ref += (g.double() * a / torch.sqrt((a * a).mean(-1, keepdim=True) + 1e-6)).sum((0, 1))
    e = float((got - ref).norm() / ref.norm()) / U
    assert e <= 3.2, e
    assert fb.fa_back_get_error() == 0


def test_weights_gradient_of_an_infinity(fb):
    """An infinite gradient component makes that of its weight infinite, of the definition's sign, and no other."""
    N, H, D = 3000, 2, 128
    rng = np.random.default_rng(91)
    (x, xa), (g, _) = act_array(rng, (N, H, D), "f32"), act_array(rng, (N, H, D), "f32")
    g[1234, 1, 17] = float("inf")
    got = fb.qk_norm_rope_backward(g, None, x, None, None, wq=torch.ones(D, device="cuda"))["dwq"].cpu().numpy()
    assert got[17] == np.sign(xa[1234, 1, 17]) * np.inf and np.isfinite(np.delete(got, 17)).all()


@pytest.mark.parametrize("sinks", [False, True])
@pytest.mark.parametrize("lens", [[500, 30], [9000, 1, 2]])
def test_f32_values_near_the_top_of_their_range(fb, lens, sinks):
    """O lies between the values, so finite values give a finite O: no weight on the way is above one."""
    p = R.Paged(101, lens, 2, 128, 128, F16, F32, 16, v_amp=1e36)
    check_decode(fb, p, 8, sinks=sinks)


@pytest.mark.parametrize("cap", [1e-45, 1e-40, 1e-38, 3e38])
def test_soft_cap_at_the_ends_of_its_range(fb, cap):
    """Caps whose reciprocal leaves f32's range, with scores that are zero (of keys of zeros) and others."""
    p = R.Paged(111, [40, 300], 2, 64, 64, F16, F16, 16)
    for b in range(2):
        j = np.arange(0, p.lens[b], 3)
        p.k[p.table[b, j // 16], j % 16] = 0
        p.kd[b][j] = 0.0
    check_decode(fb, p, 4, softcap=cap)


def test_the_marshalling_module_serves_the_plain_calls(fb, monkeypatch):
    """What test_both_forms_of_the_wrappers_agree compares is served by the module: with the Python form's entry points
    out of reach the same calls still return, and called directly none of the module's functions declines."""
    from flash_attention_backward_gb300 import _native, paged
    rng = np.random.default_rng(31)
    p = R.Paged(31, [70, 0, 200], 2, 128, 64, Q8, F16, 16)
    cache = p.on_gpu(fb, torch)
    (q, _), (k, _), (v, _) = (act_array(rng, (3, h, d), "bf16") for h, d in ((6, 128), (2, 128), (2, 64)))
    w, rope = torch.rand(128, device="cuda") + 0.5, fb.rope_frequencies(128)
    seq, pos = cuda(np.array([0, 2, 2], np.int32)), cuda(np.array([5, 17, 180], np.int32))
    lens, sinks = cuda(np.array(p.lens, np.int32)), torch.zeros(6, device="cuda")
    fb.paged_decode(q, cache, lens, scale=0.1)  # binds it

    def out_of_reach(*a):
        raise AssertionError("the Python form")

    for n in ("fa_qk_norm_rope", "fa_qk_norm_rope_backward", "fa_cache_append", "fa_cache_read", "fa_paged_decode"):
        monkeypatch.setattr(_native, n, out_of_reach)
    fb.paged_decode(q, cache, lens, scale=0.1, softcap=20.0, sinks=sinks, alibi_slopes=sinks)
    fb.cache_read(cache, seq, pos, dtype=torch.bfloat16)
    fb.cache_append(k, v, cache, seq, pos, k_norm=w, rope=rope)
    fb.qk_norm_rope(q, k, pos, wq=w, wk=w, rope=rope, rope_style=fb.FA_ROPE_PAIRS, dtype=torch.float32)
    fb.qk_norm_rope(q, None, None, wq=w)
    fb.qk_norm_rope_backward(q, k, q, k, pos, wq=w, wk=w, rope=rope)
    fb.qk_norm_rope_backward(q.float(), None, q, None, pos, rope=rope)
    f, style = paged._fast, fb.FA_ROPE_HALVES
    assert f.norm(q, k, pos, w, w, 1e-6, rope, style, None) is not None
    assert f.norm_back(q, k, q, k, pos, w, w, 1e-6, rope, style) is not None
    assert f.append(k, v, cache._at, cache._index, seq, pos, w, 1e-6, rope, style) is True
    assert f.read(cache._at, cache._index, seq, pos, torch.float16) is not None
    assert f.decode(q, cache._at, cache._index, lens, 0.1, None, 0.0, None) is not None
    with pytest.raises(AssertionError, match="the Python form"):  # (and what it declines goes there)
        fb.paged_decode(q, cache, lens, scale=0.1, workspace=fb.Workspace("cuda"))
    assert fb.fa_back_get_error() == 0
