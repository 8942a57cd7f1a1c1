"""64-bit forms of the fa_paged.h operators in numpy, and paged caches to test them on.  They share
nothing with the library; cache rows are decoded by the oracle's dequantizer."""
import math

import numpy as np

import oracle
import synth

ACT_EPS = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}  # half a step relative to the value (bf16: a whole binade's)


def rotate(x, pos, n_rot, base, halves, sign=1.0):
    """x [N][heads][D] rotated by pos [N] (float64)."""
    y = x.astype(np.float64).copy()
    i = np.arange(n_rot // 2)
    a = sign * pos.astype(np.float64)[:, None] * base ** (-2.0 * i / n_rot)
    c, s = np.cos(a)[:, None, :], np.sin(a)[:, None, :]
    first, second = (i, i + n_rot // 2) if halves else (2 * i, 2 * i + 1)
    u, v = y[..., first].copy(), y[..., second].copy()
    y[..., first], y[..., second] = u * c - v * s, u * s + v * c
    return y


def norm(x, w, eps):
    x = x.astype(np.float64)
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w.astype(np.float64)


def stored(x, t):
    """(codes or None, values) of float64 rows [..., D] stored in cache type t; the block formats' definition."""
    if t == synth.TYPE_F32:
        return None, x.astype(np.float32).astype(np.float64)
    if t == synth.TYPE_F16:
        return None, x.astype(np.float16).astype(np.float64)
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    mag = np.abs(b)
    top = mag.max(-1, keepdims=True)
    safe = np.where(top > 0, top, 1.0)
    if t == synth.TYPE_Q8_0:
        d = top / 127.0
        c = np.copysign(np.floor(mag * 127.0 / safe + 0.5), b)
    else:
        m = np.take_along_axis(b, mag.argmax(-1)[..., None], -1)  # argmax: the first of equals
        d = m / -8.0
        c = np.minimum(np.floor(np.where(top > 0, -8.0 * b / np.where(top > 0, m, 1.0), 0.0) + 8.5), 15.0) - 8.0
    d16 = d.astype(np.float32).astype(np.float16).astype(np.float64)
    return c.reshape(x.shape), (c * d16).reshape(x.shape)


class Paged:
    """A paged cache with seeded content.  Rows that no sequence holds, and the rows behind a sequence's
    length, are 0xFF bytes: NaN in every float format and in every block scale."""

    def __init__(self, seed, lens, Hkv, D, Dv, kt, vt, page, spare=3, k_amp=1.0, v_amp=1.0):
        rng = np.random.default_rng(seed)
        self.lens, self.Hkv, self.D, self.Dv, self.kt, self.vt, self.page = list(lens), Hkv, D, Dv, kt, vt, page
        B = len(self.lens)
        self.max_pages = max(1, max((-(-n // page) for n in self.lens), default=1))
        n_pages = B * self.max_pages + spare
        self.table = rng.permutation(n_pages)[: B * self.max_pages].reshape(B, self.max_pages).astype(np.int32)
        self.k = np.full((n_pages, page, Hkv, synth.row_bytes(kt, D)), 0xFF, np.uint8)
        self.v = np.full((n_pages, page, Hkv, synth.row_bytes(vt, Dv)), 0xFF, np.uint8)
        self.kd, self.vd = [], []  # decoded, per sequence
        for b, n in enumerate(self.lens):
            n = max(n, 0)
            rk = synth.quantize_rows((k_amp * rng.standard_normal((n, Hkv, D))).astype(np.float32), kt)
            rv = synth.quantize_rows((v_amp * rng.standard_normal((n, Hkv, Dv))).astype(np.float32), vt)
            j = np.arange(n)
            self.k[self.table[b, j // page], j % page] = rk
            self.v[self.table[b, j // page], j % page] = rv
            self.kd.append(oracle.dequant(rk, kt, D).reshape(n, Hkv, D) if n else np.zeros((0, Hkv, D)))
            self.vd.append(oracle.dequant(rv, vt, Dv).reshape(n, Hkv, Dv) if n else np.zeros((0, Hkv, Dv)))

    def on_gpu(self, fb, torch):
        k, v = torch.from_numpy(self.k).cuda(), torch.from_numpy(self.v).cuda()
        return fb.PagedCache(k, self.kt, v, self.vt, torch.from_numpy(self.table).cuda(), D=self.D, Dv=self.Dv)


def decode(p, q, scale, softcap=0.0, alibi=None, sinks=None):
    """O, lse and the error scale of each (see tolerance()) for queries q [B][H][D]."""
    B, H, _ = q.shape
    G = H // p.Hkv
    O, lse = np.zeros((B, H, p.Dv)), np.full((B, H), -np.inf)
    mag, smag = np.zeros((B, H, p.Dv)), np.zeros((B, H))
    for b, n in enumerate(p.lens):
        if n <= 0 and sinks is not None:
            lse[b] = sinks
        if n <= 0:
            continue
        for h in range(H):
            k, v, qq = p.kd[b][:, h // G], p.vd[b][:, h // G], q[b, h].astype(np.float64)
            x = scale * (k @ qq)
            smag[b, h] = (abs(scale) * (np.abs(k) @ np.abs(qq))).max()
            if softcap > 0:
                x = softcap * np.tanh(x / softcap)
            if alibi is not None:
                x = x + float(alibi[h]) * (np.arange(n) - (n - 1))
                smag[b, h] += abs(float(alibi[h])) * n
            every = x if sinks is None else np.append(x, float(sinks[h]))
            top = every.max()
            lse[b, h] = top + math.log(np.exp(every - top).sum())
            w = np.exp(x - lse[b, h])
            O[b, h] = w @ v
            mag[b, h] = w @ np.abs(v)
            smag[b, h] = max(smag[b, h], abs(lse[b, h]))
    return O, lse, mag, smag


def decode_tolerance(p, mag, smag, act):
    """Bounds of |O - ref| and |lse - ref|, by the roundings of an f32 computation (u = 2^-24):
    a score is a sum of D products held to (D / 16 + 24) u of the sum of magnitudes A = smag (16-term
    steps of the tensor core, block scales, q in two parts of 22 bits, and the steps behind the sum), its
    exponential is off by that and 8 u; the weights times block scales are held to 2^-17 (two bf16
    parts); a sum over n keys takes n / 16 + 64 f32 steps."""
    u = 2.0 ** -24
    n = max(max(p.lens), 1)
    ds = (p.D / 16 + 24) * u * smag
    rel = 2.0 * ds + 2.0 ** -17 + (n / 16 + 96) * u
    tol_O = rel[..., None] * mag
    tol_lse = ds + (n / 16 + 96) * u + 4 * u * smag
    return tol_O, tol_lse
