"""64-bit numpy (and list) forms of the fa_paged_ext.h operators.  They share nothing with the library."""
import numpy as np

f32 = np.float32


def rotate_axes(x, pos, axis, base, halves, sign=1.0):
    """x [N][heads][D] with pair i turned by pos[axis[i]] (pos [A][N])."""
    y = x.astype(np.float64).copy()
    n_rot = 2 * len(axis)
    i = np.arange(len(axis))
    a = sign * pos.astype(np.float64)[axis].T * base ** (-2.0 * i / max(n_rot, 1))
    c, s = np.cos(a)[:, None, :], np.sin(a)[:, None, :]
    first, second = (i, i + n_rot // 2) if halves else (2 * i, 2 * i + 1)
    u, v = y[..., first].copy(), y[..., second].copy()
    y[..., first], y[..., second] = u * c - v * s, u * s + v * c
    return y


class Lists:
    """Page lists as Python lists, request by request."""

    def __init__(self, table, lens, stack, num_pages, page):
        self.table, self.lens, self.stack, self.num_pages, self.page = table.tolist(), list(lens), list(stack), num_pages, page

    def extend(self, news, T):
        p, width = self.page, len(self.table[0])
        starts, first, seq, pos, row = [0], [], [], [], []
        asked, room = 0, len(self.stack)
        for b, (n, m) in enumerate(zip(list(self.lens), news)):
            m = max(m, 0) if n >= 0 else 0
            begin = starts[-1] if b == 0 else end
            end = begin + m
            good = m > 0 and n + m <= width * p and end <= T
            need = -(-(n + m) // p) - -(-n // p) if good else 0
            asked += need
            good = good and (need == 0 or asked <= room)
            if good:
                for i in range(need):
                    self.table[b][-(-n // p) + i] = self.stack.pop()
                self.lens[b] = n + m
            first.append(n if good else -1)
            for i in range(min(m, max(0, T - begin))):
                seq.append(b if good else -1)
                pos.append(n + i if good else -1)
                row.append(self.table[b][(n + i) // p] * p + (n + i) % p if good else -1)
            starts.append(min(end, T))
        for x in (seq, pos, row):
            x += [-1] * (T - len(x))
        return dict(seq=seq, pos=pos, row=row, starts=starts, first=first)

    def trim(self, keep):
        p = self.page
        for b in reversed(range(len(self.lens))):
            n, k = self.lens[b], keep[b]
            if k < 0 or k >= n:
                continue
            for j in reversed(range(-(-k // p), -(-n // p))):
                self.stack.append(self.table[b][j])
                self.table[b][j] = -1
            self.lens[b] = k


def bounds(rows):
    """codes [2][D] and scales [D / 32] of a page's key values rows [n][D] (f64)."""
    hi, lo = (x.astype(f32).reshape(-1, 32) for x in (rows.max(0), rows.min(0)))
    m = np.maximum(abs(hi), abs(lo)).max(1, keepdims=True)
    some = m > f32(1e-30)
    d = np.where(some, m / f32(127), f32(0)).astype(f32)
    safe = np.where(some, d, f32(1))
    up = np.clip(np.ceil((hi / safe).astype(f32)), -127, 127) * some
    down = np.clip(np.floor((lo / safe).astype(f32)), -127, 127) * some
    return np.stack([up.ravel(), down.ravel()]).astype(np.int8), d[:, 0]


def score(q, codes, scales, scale, far=None, slope=None):
    """The f32 score of pages codes [n][2][D], scales [n][D / 32] for one query head q [D] (f32)."""
    q = q.astype(f32).reshape(-1, 32)
    m = abs(q).max(1, keepdims=True)
    some = m > f32(1e-30)
    safe = np.where(some, m, f32(1))
    c = np.clip(np.rint(q * (f32(127) / safe)), -127, 127) * some
    e = (m / f32(127) * some)[:, 0].astype(f32)
    c = c.astype(np.int64)
    n = len(codes)
    hi, lo = (codes[:, k].astype(np.int64).reshape(n, -1, 32) for k in (0, 1))
    I = np.where(c > 0, c * hi, c * lo).sum(-1)
    t = (I.astype(f32) * scales) * e
    assert t.dtype == f32
    while t.shape[1] > 1:
        t = t[:, ::2] + t[:, 1::2]
    s = t[:, 0] * f32(scale)
    if slope is not None:
        s = s + f32(slope) * far.astype(f32)
    assert s.dtype == f32
    return s


def select(q, codes, scales, n_pages, L, page, G, K, scale, first, last, slopes=None):
    """Chosen pages of one KV head: q [G][D], codes / scales of its n_pages pages in their order."""
    if n_pages <= K:
        return list(range(n_pages))
    j = np.arange(n_pages)
    far = np.minimum((j + 1) * page, L) - L
    best = np.full(n_pages, -np.inf, f32)
    for g in range(G):
        s = score(q[g], codes, scales, scale, far, None if slopes is None else slopes[g])
        best = np.maximum(best, np.where(np.isnan(s), f32(np.inf), s))
    must = (j < first) | (j >= n_pages - last)
    order = sorted(range(n_pages), key=lambda i: (not must[i], -float(best[i]), i))
    return sorted(order[:K])
