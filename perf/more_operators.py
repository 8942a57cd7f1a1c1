"""Positions of several axes, page lists and attention over selected pages: cases, plain forms and 64-bit values.

Operators
  axes       RMS norm of every query and key head and the rotation by positions of several axes (qk_norm_rope with
             rope_axes: time, height, width of images and video)
  axes_back  the gradient of that with respect to q, k and both norm weights (qk_norm_rope_backward)
  store      keys (normalised, rotated by several axes) and values into a paged raw cache (cache_append); the rows
             are then read back decoded (cache_read)
  pages      page tables and the slots of the new tokens, made on the GPU from the requests' lengths (pages_extend);
             then the tokens are given up again, as drafts that were rejected (pages_trim)
  bounds     the largest and the smallest component of each page's keys, in 8 bits (page_bounds)
  sparse     the pages whose bounds promise the largest scores are chosen for each query (page_select), and one new
             token per sequence attends over them (paged_decode with pages)

Cache rows: f32 and f16 values; q8_0 blocks of 32 (binary16 scale d, 32 int8 codes, value code * d);
q4_0 blocks of 32 (binary16 scale d, 16 bytes, byte b holding element b low and b + 16 high, value
(nibble - 8) * d).  A pool is [num_pages][page_size][Hkv][row bytes]; position j of sequence b is row
j % page_size of page page_table[b][j // page_size].

Rotation: pair i of a head of token n turns by pos[axis[i]][n] * inv_freq[i].

Bounds of a page and KV head: over its rows that are there, per component, hi = max and lo = min; in blocks of 32
d = fl(max(|hi|, |lo|) / 127), codes ceil(fl(hi / d)) and floor(fl(lo / d)) within +-127 (zeros where no value is above
1e-30).  Score of a page for query head h: q in blocks of 32, m = max |q|, codes c = round(fl(q * fl(127 / m))), ties to
even, within +-127, e = fl(m / 127) (zeros where m <= 1e-30); I = sum of c * hi where c > 0 and c * lo elsewhere;
the sum of the terms fl(fl(I * d) * e) over the blocks, neighbours first (a tree); times scale; plus
fl(slope * distance of the page's last key); each step rounded to f32 (fl).  A KV head's score is the largest of its
query heads'.  Chosen: the first and the last pages asked for, then the largest scores, ties to the lowest page.
"""
import math

import torch

own = False

ROW = {"f32": lambda D: 4 * D, "f16": lambda D: 2 * D, "q8_0": lambda D: D // 32 * 34, "q4_0": lambda D: D // 32 * 18}
CODE = {"f32": 0, "f16": 1, "q8_0": 2, "q4_0": 3}
ACT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ACT_BYTES = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-6
TINY = 1e-30


# ------------------------------------------------------------------------------------------------
# cases

def _axes(name, op, N, H, Hkv, D, act, out, sections, interleaved, halves, fused, start):
    return {"name": name, "op": op, "N": N, "H": H, "Hkv": Hkv, "D": D, "act": act, "out": out, "sections": sections,
            "interleaved": interleaved, "halves": halves, "fused": fused, "start": start}


def _store(name, T, B, start, Hkv, D, kt, vt, act, page, sections, interleaved, halves, k_norm):
    return {"name": name, "op": "store", "T": T, "B": B, "start": start, "Hkv": Hkv, "D": D, "kt": kt, "vt": vt, "act": act,
            "page": page, "sections": sections, "interleaved": interleaved, "halves": halves, "k_norm": k_norm}


def _pages_case(name, B, new, page, max_len, short):
    return {"name": name, "op": "pages", "B": B, "new": new, "page": page, "max_len": max_len, "short": short}


def _bounds(name, B, max_len, lens, news, Hkv, D, kt, page):
    return {"name": name, "op": "bounds", "B": B, "max_len": max_len, "lens": lens, "news": news, "Hkv": Hkv, "D": D, "kt": kt,
            "page": page}


def _sparse(name, B, max_len, lens, H, Hkv, D, kt, vt, act, page, K, first, last, softcap=0.0, alibi=False, sinks=False):
    return {"name": name, "op": "sparse", "B": B, "max_len": max_len, "lens": lens, "H": H, "Hkv": Hkv, "D": D, "kt": kt,
            "vt": vt, "act": act, "page": page, "K": K, "first": first, "last": last, "softcap": softcap, "alibi": alibi,
            "sinks": sinks}


def listed():
    return [
        # a decode step's queries and keys of a model that saw images: three axes
        _axes("axes_step_bf16", "axes", 64, 32, 8, 128, "bf16", "bf16", "16,24,24", False, True, True, 9000),
        # a piece of a video prompt at the long-context shape, in the f32 that the attention takes, axes in turn
        _axes("axes_video_f32", "axes", 2048, 24, 4, 256, "f32", "f32", "44,42,42", True, True, False, 73472),
        # training on images: two axes, half of each head rotated, neighbouring pairs
        _axes("axes_back_f32", "axes_back", 2048, 24, 4, 256, "f32", "f32", "32,32", False, False, False, 0),
        # training in 16-bit activations with an odd token count
        _axes("axes_back_bf16", "axes_back", 8191, 32, 8, 128, "bf16", "bf16", "24,20,20", True, True, True, 0),
        # a decode step's new rows: one token for each of 64 sequences
        _store("store_step_q8", 64, 64, 4000, 4, 256, "q8_0", "q8_0", "f32", 64, "44,42,42", True, True, True),
        # image prompts of several sequences in one call, mixed types
        _store("store_ragged_mixed", 5003, 7, 11, 8, 128, "f16", "q4_0", "bf16", 16, "16,24,24", False, True, True),
        # a decode step: one token for each of 64 requests
        _pages_case("pages_step", 64, "one", 64, 8192, False),
        # prompts coming in beside running requests, and not enough pages for all of them
        _pages_case("pages_prompts_short", 509, "prompts", 16, 4096, True),
        # a decode step: the page that each of 64 sequences is writing to
        _bounds("bounds_step_q8", 64, 512, "ragged", "one", 4, 256, "q8_0", 64),
        # a whole prompt of the benchmark's length
        _bounds("bounds_prompt_q8", 1, 75520, "full", "all", 4, 256, "q8_0", 64),
        # one sequence at the long-context length of the benchmark, 64 of its 1180 pages
        _sparse("sparse_long_q8", 1, 75520, "full", 24, 4, 256, "q8_0", "q8_0", "f32", 64, 64, 1, 2),
        # a serving batch of unequal lengths, some slots empty, binary16 cache, small pages
        _sparse("sparse_batch_f16", 48, 8192, "ragged", 32, 8, 128, "f16", "f16", "bf16", 16, 64, 1, 4, 0.0, False, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _sections(rng, D, halves):
    """Pairs of each axis: two to four axes over the whole head or a half of it."""
    pairs = rng.choice([D // 2, D // 4])
    A = rng.choice([2, 3, 3, 4])
    cut = sorted(rng.sample(range(1, pairs), A - 1))
    return ",".join(str(b - a) for a, b in zip([0] + cut, cut + [pairs]))


def draw(rng):
    op = rng.choice(["axes", "axes_back", "store", "pages", "bounds", "sparse"])
    D = rng.choice([64, 128, 256])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    types = ["f32", "f16", "q8_0", "q4_0"]
    act = rng.choice(["f32", "f16", "bf16"])
    halves = rng.random() < 0.6
    page = rng.choice([16, 32, 40, 48, 64, 128, 256])
    if op in ("axes", "axes_back"):
        H = Hkv * rng.choice([1, 2, 3, 4, 6, 8])
        N = _log(rng, 1, min(20000, 30000000 // ((H + Hkv) * D)))
        return _axes("", op, N, H, Hkv, D, act, act if op == "axes_back" else rng.choice([act, "f32"]), _sections(rng, D, halves),
                     rng.random() < 0.5, halves, rng.random() < 0.5, rng.randrange(0, 1000000))
    if op == "store":
        T = _log(rng, 1, min(8192, 12000000 // (Hkv * D)))
        return _store("", T, min(T, _log(rng, 1, 64)), rng.randrange(0, 100000), Hkv, D, rng.choice(types), rng.choice(types),
                      act, rng.choice([16, 32, 48, 64, 128]), _sections(rng, D, halves), rng.random() < 0.5, halves, rng.random() < 0.6)
    if op == "pages":
        return _pages_case("", _log(rng, 1, 509), rng.choice(["one", "drafts", "prompts"]), rng.choice([1, 5, 16, 32, 64, 100, 256]),
                           _log(rng, 64, 4096), rng.random() < 0.3)
    kt = rng.choice(types)
    B = _log(rng, 1, 96)
    if op == "bounds":
        top = int(80e6 / (B * Hkv * ROW[kt](D)))
        return _bounds("", B, _log(rng, 1, max(1, min(75520, top))), rng.choice(["full", "ragged"]), rng.choice(["one", "some", "all"]),
                       Hkv, D, kt, page)
    G = rng.choice([1, 2, 3, 4, 6, 8, 12])
    vt = rng.choice(types)
    top = int(200e6 / (B * Hkv * (ROW[kt](D) + ROW[vt](D))))
    K = rng.choice([4, 8, 16, 33, 64])
    return _sparse("", B, _log(rng, 1, max(1, min(75520, top))), rng.choice(["full", "ragged"]), G * Hkv, Hkv, D, kt, vt, act, page, K,
                   rng.choice([0, 1, 2]), rng.choice([0, 1, 2]), rng.choice([0.0, 0.0, 30.0, 50.0]), rng.random() < 0.3, rng.random() < 0.3)


def _lens(case):
    """The sequences' lengths: part of the case.  Ragged ones spread over the whole range (a golden-ratio
    sequence, cubed half of the time), with every eighth slot empty and one of length one."""
    if case["lens"] == "full":
        return [case["max_len"]] * case["B"]
    out = []
    for b in range(case["B"]):
        u = (0.5 + 0.6180339887498949 * b) % 1.0
        u = u ** 3 if b % 2 else u
        out.append(0 if b % 8 == 5 else 1 if b == 3 else max(1, int(round(u * case["max_len"]))))
    out[0] = case["max_len"]
    return out


def _firsts(case, lens):
    """The first position of each sequence that is new since its bounds were last computed; -1: none is."""
    news = {"one": lambda n: n - 1, "some": lambda n: n - 1 - n // 3, "all": lambda n: 0}[case["news"]]
    return [news(n) if n else -1 for n in lens]


def _split(case):
    """(sequence, position) of each stored token: the sequences' shares are unequal."""
    T, B = case["T"], case["B"]
    w = [1.0 + (0.6180339887498949 * b) % 1.0 for b in range(B)]
    n = [max(1, int(T * x / sum(w))) for x in w]
    n[0] += T - sum(n)
    if n[0] < 1:
        n = [T // B + (b < T % B) for b in range(B)]
    seq, pos = [], []
    for b in range(B):
        first = case["start"] + 13 * b
        seq += [b] * n[b]
        pos += range(first, first + n[b])
    return seq, pos


def _requests(case):
    """(length, new tokens) of each request: a sixteenth of the slots are free (-1), some requests have nothing new."""
    B, top = case["B"], case["max_len"]
    lens, news = [], []
    for b in range(B):
        u, v = (0.5 + 0.6180339887498949 * b) % 1.0, (0.3 + 0.7548776662466927 * b) % 1.0
        if case["new"] == "prompts":
            n = max(1, int(v * v * top / 4)) if b % 3 else 1
        else:
            n = 1 if case["new"] == "one" else 1 + int(v * 8)
        lens.append(-1 if b % 16 == 7 else 0 if case["new"] == "prompts" and b % 3 else int(u * max(0, top - n)))
        news.append(0 if b % 16 == 11 else n)
    return lens, news


def _page_need(case):
    """Pages that the requests hold, and that they ask for."""
    lens, news = _requests(case)
    p, held, asked = case["page"], 0, 0
    for n, m in zip(lens, news):
        if n >= 0:
            held += -(-n // p)
            asked += -(-(n + m) // p) - -(-n // p)
    return held, asked


def work(case):
    if case["op"] == "pages":
        lens, news = _requests(case)
        T, (held, asked) = sum(m for n, m in zip(lens, news) if n >= 0), _page_need(case)
        # lengths, new ones and starts; the tokens' sequence, position and row; table entries and stack entries, there and back
        return {"bytes": 4 * (6 * case["B"] + 3 * T + 4 * asked), "flops": 4 * T + 20 * case["B"]}
    D, Hkv = case["D"], case["Hkv"]
    if case["op"] == "bounds":
        lens, p = _lens(case), case["page"]
        pages = rows = 0
        for n, f in zip(lens, _firsts(case, lens)):
            if n and f >= 0:
                pages += -(-n // p) - f // p
                rows += n - f // p * p
        return {"bytes": Hkv * (rows * ROW[case["kt"]](D) + pages * (2 * D + D // 8)), "flops": 3 * rows * Hkv * D}
    a = ACT_BYTES[case["act"]]
    if case["op"] == "sparse":
        lens, p, H = _lens(case), case["page"], case["H"]
        pages = sum(-(-n // p) for n in lens)
        rows = sum(min(n, case["K"] * p) for n in lens)
        return {"bytes": pages * Hkv * (2 * D + D // 8) + rows * Hkv * (ROW[case["kt"]](D) + ROW[case["vt"]](D))
                + 2 * case["B"] * H * D * a + 4 * case["B"] * (H + Hkv * case["K"]), "flops": 2 * H * D * pages + 4 * H * D * rows}
    if case["op"] == "store":
        rows = case["T"] * Hkv
        raw = ROW[case["kt"]](D) + ROW[case["vt"]](D)
        # new rows read and stored; the stored rows read and given out in binary16
        return {"bytes": rows * (2 * D * a + 2 * raw + 2 * D * 2), "flops": rows * D * 12}
    rows, o = case["N"] * (case["H"] + Hkv), ACT_BYTES[case["out"]]
    if case["op"] == "axes":
        return {"bytes": rows * D * (a + o), "flops": rows * D * 9}
    return {"bytes": rows * D * (a + o + a) + 4 * D * 4, "flops": rows * D * 20}


# ------------------------------------------------------------------------------------------------
# inputs

def _quantise(x, t):
    """Rows of a type from float values [..., D], as bytes.  The block scale is amax / 127 (q8_0) or the value of
    largest magnitude / -8 (q4_0), stored in binary16; codes are the nearest to value / scale, ties away from zero
    (q8_0) or up (q4_0)."""
    if t == "f32":
        return x.to(torch.float32).contiguous().view(torch.uint8)
    if t == "f16":
        return x.to(torch.float16).contiguous().view(torch.uint8)
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    if t == "q8_0":
        top = b.abs().amax(-1, keepdim=True)
        d = top / 127
        y = torch.where(top > 0, b * 127 / torch.where(top > 0, top, 1), 0)  # one rounding: half of the largest is a tie
        c = torch.trunc(y + torch.copysign(torch.full_like(y, 0.5), y)).clamp(-127, 127).to(torch.int8).view(torch.uint8)
    else:
        mag = b.abs()
        at = torch.where(mag == mag.amax(-1, keepdim=True), torch.arange(32, device=x.device), 31).amin(-1, keepdim=True)  # the first of equals
        d = b.gather(-1, at) / -8
        y = torch.where(d != 0, b / torch.where(d != 0, d, 1), 0)
        n = torch.floor(y + 8.5).clamp(0, 15).to(torch.uint8)
        c = n[..., :16] | (n[..., 16:] << 4)
    d16 = d.to(torch.float32).to(torch.float16).view(torch.uint8)
    return torch.cat([d16, c], -1).flatten(-2)


def _decoded(raw, t, kind):
    """The values of rows of bytes [..., row], in the type `kind`."""
    if t == "f32":
        return raw.contiguous().view(torch.float32).to(kind)
    if t == "f16":
        return raw.contiguous().view(torch.float16).to(kind)
    blk = raw.unflatten(-1, (-1, 34 if t == "q8_0" else 18))
    d = blk[..., :2].contiguous().view(torch.float16).to(kind)
    if t == "q8_0":
        c = blk[..., 2:].contiguous().view(torch.int8).to(kind)
    else:
        c = torch.cat([blk[..., 2:] & 15, blk[..., 2:] >> 4], -1).to(kind) - 8
    return (c * d).flatten(-2)


def _rope(n_rot, base, dev):
    """inv_freq in 64 bits, and the same as turns per position in units of 2^-64 (the framework's form)."""
    inv = [base ** (-2.0 * i / n_rot) for i in range(n_rot // 2)]
    fixed = [int(f / (2.0 * math.pi) * 2.0 ** 64) for f in inv]
    return torch.tensor(inv, dtype=torch.float64, device=dev), torch.tensor(fixed, dtype=torch.int64, device=dev)


def _axis_of_pairs(case):
    """The axis of each pair: the sections one after another, or in turn while they last."""
    left = [int(n) for n in case["sections"].split(",")]
    if not case["interleaved"]:
        return [a for a, n in enumerate(left) for _ in range(n)]
    out = []
    while any(left):
        for a in range(len(left)):
            if left[a]:
                left[a] -= 1
                out.append(a)
    return out


def _grid(start, N, A, dev):
    """Positions [A][N] of a video's patches behind `start` tokens of text: frames of 24 by 42 patches; the first
    sixteenth of the tokens is text, whose positions are the same on every axis."""
    i = torch.arange(N, device=dev)
    text = N // 16
    j = (i - text).clamp_min(0)
    grid = torch.stack([j // (24 * 42), j // 42 % 24, j % 42, j % 7])[:A] + start + text
    return torch.where(i < text, start + i, grid).to(torch.int32).contiguous()


def _pages(gen, B, max_pages, dev):
    n = B * max_pages + 3
    return n, torch.randperm(n, generator=gen, device=dev)[: B * max_pages].reshape(B, max_pages).to(torch.int32)


def _pool(gen, n_rows, Hkv, D, t, dev, spread=None):
    out = torch.empty((n_rows, Hkv, ROW[t](D)), dtype=torch.uint8, device=dev)
    step = max(1, (1 << 25) // (Hkv * D))
    for r in range(0, n_rows, step):
        m = min(step, n_rows - r)
        x = torch.randn((m, Hkv, D), generator=gen, device=dev)
        out[r:r + m] = _quantise(x if spread is None else x * spread, t)
    return out


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    s = {"case": case}

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    if case["op"] == "pages":
        B, p = case["B"], case["page"]
        lens, news = _requests(case)
        held, asked = _page_need(case)
        spare = asked // 2 if case["short"] else asked + 5
        width = -(-max(n + m for n, m in zip(lens, news)) // p)
        width = max(1, width - (1 if case["short"] else 0))  # (the longest request does not fit the table then)
        lens = [min(n, width * p) for n in lens]
        num_pages = held + spare
        order = torch.randperm(num_pages, generator=gen, device=dev).to(torch.int32)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        s["news"] = torch.tensor(news, dtype=torch.int32, device=dev)
        count = (s["lens"].clamp_min(0) + p - 1) // p
        first = torch.cumsum(count, 0) - count
        j = torch.arange(width, device=dev)
        s["table"] = torch.where(j < count[:, None], order[(first[:, None] + j).clamp_max(num_pages - 1)], -1).to(torch.int32)
        used = int(count.sum())
        s["free"] = torch.full((num_pages,), -1, dtype=torch.int32, device=dev)
        s["free"][: num_pages - used] = order[used:]
        s["num_free"] = torch.tensor([num_pages - used], dtype=torch.int32, device=dev)
        s["T"] = sum(m for n, m in zip(lens, news) if n >= 0) + 3
        s["keep"] = s["lens"].clone()
        if own:
            import flash_attention_backward_gb300 as fb
            s["lists"] = fb.PageLists(s["table"], s["lens"], s["free"], s["num_free"], page_size=p)
        return s
    D, Hkv = case["D"], case["Hkv"]
    if case["op"] in ("sparse", "bounds"):
        B, page = case["B"], case["page"]
        max_pages = -(-case["max_len"] // page)
        n_pages, s["table"] = _pages(gen, B, max_pages, dev)
        # keys as a model's: some components are several times as large as the others
        spread = torch.exp(0.7 * normal(Hkv, D))
        s["k"] = _pool(gen, n_pages * page, Hkv, D, case["kt"], dev, spread).view(n_pages, page, Hkv, -1)
        s["lens"] = torch.tensor(_lens(case), dtype=torch.int32, device=dev)
        s["codes"] = torch.zeros((n_pages, Hkv, 2, D), dtype=torch.int8, device=dev)
        s["scales"] = torch.zeros((n_pages, Hkv, D // 32), dtype=torch.float32, device=dev)
        vt = case.get("vt", case["kt"])
        if case["op"] == "bounds":
            s["v"] = s["k"]
            s["first"] = torch.tensor(_firsts(case, _lens(case)), dtype=torch.int32, device=dev)
        else:
            H = case["H"]
            s["v"] = _pool(gen, n_pages * page, Hkv, D, vt, dev).view(n_pages, page, Hkv, -1)
            s["q"] = normal(B, H, D).to(ACT[case["act"]])
            s["scale"] = D ** -0.5
            s["alibi"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], device=dev) if case["alibi"] else None
            s["sinks"] = 1.0 + normal(H) if case["sinks"] else None
            s["first"] = None
            _plain_bounds(s)
        if own:
            import flash_attention_backward_gb300 as fb
            s["cache"] = fb.PagedCache(s["k"], CODE[case["kt"]], s["v"], CODE[vt], s["table"], D=D, Dv=D)
            s["bounds"] = fb.PageBounds(s["codes"], s["scales"])
        return s
    axis = _axis_of_pairs(case)
    s["axis"] = torch.tensor(axis, dtype=torch.uint8, device=dev)
    act, A = ACT[case["act"]], len(case["sections"].split(","))
    if case["op"] == "store":
        T, B, page = case["T"], case["B"], case["page"]
        seq, pos = _split(case)
        max_pages = max(pos) // page + 1
        # the table is as wide as the positions ask for; pages are shared out to those that this call stores into
        width = max_pages - min(pos) // page
        n_pages, small = _pages(gen, B, width, dev)
        s["table"] = torch.zeros((B, max_pages), dtype=torch.int32, device=dev)
        s["table"][:, max_pages - width:] = small
        s["seq"] = torch.tensor(seq, dtype=torch.int32, device=dev)
        s["pos"] = torch.tensor(pos, dtype=torch.int32, device=dev)
        s["axes_pos"] = _grid(case["start"] // 3, T, A, dev)
        s["k"] = torch.zeros((n_pages, page, Hkv, ROW[case["kt"]](D)), dtype=torch.uint8, device=dev)
        s["v"] = torch.zeros((n_pages, page, Hkv, ROW[case["vt"]](D)), dtype=torch.uint8, device=dev)
        s["xk"], s["xv"] = normal(T, Hkv, D).to(act), normal(T, Hkv, D).to(act)
        s["wk"] = 1.0 + 0.1 * normal(D) if case["k_norm"] else None
        s["inv_freq"], s["rope"] = _rope(2 * len(axis), 10000.0, dev)
        if own:
            import flash_attention_backward_gb300 as fb
            s["cache"] = fb.PagedCache(s["k"], CODE[case["kt"]], s["v"], CODE[case["vt"]], s["table"], D=D, Dv=D)
        return s
    N, H = case["N"], case["H"]
    x = normal(N, H + 2 * Hkv, D).to(act) if case["fused"] else None  # one projection of q, k and v
    s["q"] = x[:, :H] if case["fused"] else normal(N, H, D).to(act)
    s["k"] = x[:, H:H + Hkv] if case["fused"] else normal(N, Hkv, D).to(act)
    s["axes_pos"] = _grid(case["start"], N, A, dev)
    s["wq"], s["wk"] = 1.0 + 0.1 * normal(D), 1.0 + 0.1 * normal(D)
    s["inv_freq"], s["rope"] = _rope(2 * len(axis), 1000000.0, dev)
    if case["op"] == "axes_back":
        s["gq"], s["gk"] = normal(N, H, D).to(ACT[case["out"]]), normal(N, Hkv, D).to(ACT[case["out"]])
    return s


# ------------------------------------------------------------------------------------------------
# the plain forms

def _turned(x, cos, sin, halves, back):
    """x [..., D] with its first 2 * pairs components rotated by the angles whose cos / sin [..., pairs] are given."""
    h = cos.shape[-1]
    if back:
        sin = -sin
    if halves:
        a, b = x[..., :h], x[..., h:2 * h]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = x[..., 0:2 * h:2], x[..., 1:2 * h:2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([y, x[..., 2 * h:]], -1)


def _angles(s, kind):
    a = s["axes_pos"][s["axis"].long()].t().to(torch.float64)[:, None] * s["inv_freq"]  # [tokens][1][pairs]
    return torch.cos(a).to(kind), torch.sin(a).to(kind)


def _normed(x, w):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w


def _plain_axes(s):
    case = s["case"]
    cos, sin = _angles(s, torch.float32)
    return {n: _turned(_normed(s[n].float(), s["w" + n]), cos, sin, case["halves"], False).to(ACT[case["out"]]) for n in ("q", "k")}


def _plain_back_of(s, n, cos, sin):
    case = s["case"]
    x, w = s[n].float(), s["w" + n]
    g = _turned(s["g" + n].float(), cos, sin, case["halves"], True)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    h = g * w
    dx = r * (h - x * (r * r * (h * x).mean(-1, keepdim=True)))
    return {"dw" + n: (g * x * r).to(torch.float64).sum((0, 1)).float(), "d" + n: dx.to(ACT[case["act"]])}


def _plain_axes_back(s):
    cos, sin = _angles(s, torch.float32)
    return {**_plain_back_of(s, "q", cos, sin), **_plain_back_of(s, "k", cos, sin)}


def _plain_store(s):
    case = s["case"]
    # 64 bits for the quantised types: a value next to a code's border must not fall on its other side
    f = torch.float64 if case["kt"] in ("q8_0", "q4_0") else torch.float32
    k = s["xk"].to(f)
    if s["wk"] is not None:
        k = _normed(k, s["wk"].to(f))
    cos, sin = _angles(s, f)
    k = _turned(k, cos, sin, case["halves"], False)
    page = s["table"][s["seq"].long(), s["pos"].long() // case["page"]].long()
    row = s["pos"].long() % case["page"]
    s["k"][page, row] = _quantise(k, case["kt"])
    s["v"][page, row] = _quantise(s["xv"].to(torch.float64), case["vt"])
    return {"k": _decoded(s["k"][page, row], case["kt"], torch.float32).to(torch.float16),
            "v": _decoded(s["v"][page, row], case["vt"], torch.float32).to(torch.float16)}


def _plain_pages(s):
    p, T, lens, table, free = s["case"]["page"], s["T"], s["lens"], s["table"], s["free"]
    B, width = table.shape
    dev = table.device
    F = s["num_free"]
    new = torch.where((lens >= 0) & (s["news"] > 0), s["news"], 0)
    end = torch.cumsum(new, 0).to(torch.int32)
    starts = torch.cat([torch.zeros(1, dtype=torch.int32, device=dev), end]).clamp_max(T)
    old = (lens.clamp_min(0) + p - 1) // p
    fits = (lens + new <= width * p) & (end <= T)
    need = torch.where(fits & (new > 0), (lens.clamp_min(0) + new + p - 1) // p - old, 0)
    upto = torch.cumsum(need, 0)
    ok = (new > 0) & fits & ((upto <= F) | (need == 0))
    # the pages, off the top of the stack in the sequences' order
    j = torch.arange(width, device=dev)
    at = F - 1 - (upto - need)[:, None] - (j - old[:, None])
    mine = ok[:, None] & (j >= old[:, None]) & (j < (old + need)[:, None])
    table.copy_(torch.where(mine, free[torch.where(mine, at, 0)], table))
    taken = torch.where(ok, need, 0)
    s["num_free"] -= taken.sum().to(torch.int32)
    # the tokens
    t = torch.arange(T, device=dev)
    begins = torch.zeros(T + 1, dtype=torch.int64, device=dev).index_add_(0, starts[1:].long(), torch.ones(B, dtype=torch.int64, device=dev))
    seq = torch.cumsum(begins[:T], 0).clamp_max(B - 1)
    there = ok[seq] & (t < starts[B])
    pos = torch.where(there, lens[seq] + t - starts[seq], -1)
    row = torch.where(there, table[seq, pos.clamp_min(0) // p] * p + pos.clamp_min(0) % p, -1)
    first = torch.where(ok, lens, -1)
    lens += torch.where(ok, new, 0)
    out = {"seq": torch.where(there, seq, -1).to(torch.int32), "pos": pos.to(torch.int32), "row": row.to(torch.int32), "starts": starts, "first": first}
    # given up again: pages behind the lengths that are kept go back, the last one taken first
    keep = torch.where(s["keep"] < 0, lens, torch.minimum(s["keep"], lens))
    kept, had = (keep.clamp_min(0) + p - 1) // p, (lens.clamp_min(0) + p - 1) // p
    back = had - kept
    total = back.sum()
    gone = (j >= kept[:, None]) & (j < had[:, None])
    at = s["num_free"] + total - 1 - (torch.cumsum(back, 0) - back)[:, None] - (j - kept[:, None])
    spot = torch.where(gone, at, free.numel()).flatten()
    free.copy_(torch.cat([free, free[:1]]).index_copy_(0, torch.where(gone.flatten(), spot, free.numel()), torch.where(gone, table, 0).flatten())[:-1])
    table.copy_(torch.where(gone, -1, table))
    s["num_free"] += total.to(torch.int32)
    lens.copy_(keep)
    return {**out, "table": table, "lens": lens, "free": free, "num_free": s["num_free"]}


def _by_127(x):
    return x / torch.full_like(x, 127.0)  # (a tensor's division: rounded, where a number's is a product)


def _plain_bounds(s):
    """Bounds of the pages from first // page on (None: from the start), in place: codes, scales; and their values."""
    case = s["case"]
    p, D, Hkv, table = case["page"], case["D"], case["Hkv"], s["table"]
    B, width = table.shape
    lens = s["lens"]
    first = torch.zeros_like(lens) if s["first"] is None else s["first"]
    j = torch.arange(width, device=lens.device)
    todo = (first >= 0)[:, None] & (j >= (first // p)[:, None]) & (j < ((lens + p - 1) // p)[:, None])
    b, pg = todo.nonzero(as_tuple=True)
    at = table[b, pg].long()
    k = _decoded(s["k"][at], case["kt"], torch.float32)  # [n][page][Hkv][D]
    there = (torch.arange(p, device=lens.device) + pg[:, None] * p < lens[b][:, None])[:, :, None, None]
    hi, lo = torch.where(there, k, -math.inf).amax(1), torch.where(there, k, math.inf).amin(1)
    hi, lo = hi.unflatten(-1, (-1, 32)), lo.unflatten(-1, (-1, 32))
    top = torch.maximum(hi.abs(), lo.abs()).amax(-1, keepdim=True)
    some = top > TINY
    d = torch.where(some, _by_127(top), 0)
    safe = torch.where(some, d, 1)
    ch = torch.where(some, torch.ceil(hi / safe).clamp(-127, 127), 0)
    cl = torch.where(some, torch.floor(lo / safe).clamp(-127, 127), 0)
    s["codes"][at] = torch.stack([ch.flatten(-2), cl.flatten(-2)], 2).to(torch.int8)
    s["scales"][at] = d[..., 0]


def _bound_values(s):
    c = s["codes"]
    return torch.mul(c.view(*c.shape[:3], -1, 32), s["scales"][:, :, None, :, None])


def _tree(x):
    """The sum over the last axis (a power of two), neighbours first."""
    x = x[..., 0::2] + x[..., 1::2]
    return _tree(x) if x.shape[-1] > 1 else x[..., 0]


def _plain_select(s):
    case = s["case"]
    B, H, Hkv, D, p, K = (case[n] for n in ("B", "H", "Hkv", "D", "page", "K"))
    G, n = H // Hkv, s["table"].shape[1]
    at, lens = s["table"].long(), s["lens"]
    q = s["q"].float().view(B, Hkv, G, D // 32, 32)
    m = q.abs().amax(-1, keepdim=True)
    some = m > TINY
    e = torch.where(some, _by_127(m), 0)
    r = torch.where(some, torch.full_like(m, 127.0) / torch.where(some, m, 1), 0)
    c = torch.round(q * r).clamp(-127, 127).transpose(2, 3)  # [B][Hkv][block][G][32]
    codes = s["codes"][at].float().unflatten(-1, (-1, 32)).permute(0, 2, 4, 3, 5, 1)  # [B][Hkv][block][2][32][n]
    # sums of 32 products of whole numbers, all below 2^24: exact in any order
    I = torch.matmul(c.clamp_min(0), codes[:, :, :, 0]) + torch.matmul(c.clamp_max(0), codes[:, :, :, 1])
    d = s["scales"][at].permute(0, 2, 3, 1)[:, :, :, None]  # [B][Hkv][block][1][n]
    x = _tree((I * d * e.transpose(2, 3)).movedim(2, -1)) * s["scale"]  # [B][Hkv][G][n]
    j = torch.arange(n, device=q.device)
    if s["alibi"] is not None:
        far = torch.minimum((j + 1) * p, lens[:, None]) - lens[:, None]
        x = x + s["alibi"].view(1, Hkv, G, 1) * far.float()[:, None, None]
    x = x.amax(2) + 0.0
    x = torch.where(x.isnan(), math.inf, x)
    count = ((lens + p - 1) // p)[:, None, None]
    must = (j < case["first"]) | (j >= count - case["last"])
    # forced pages before all others; those behind the sequence's last one after them
    rank = torch.where(j >= count, 0, torch.where(must, 2, 1)).expand(B, Hkv, n)
    order = torch.argsort(x, dim=-1, descending=True, stable=True)
    order = order.gather(-1, torch.argsort(rank.gather(-1, order), dim=-1, descending=True, stable=True))
    got = order[..., :K]
    got = torch.where(got < count, got, n)  # behind the last page: to the end
    got = torch.sort(got, -1)[0]
    pages = torch.where(got < n, got, -1)
    if n < K:
        pages = torch.cat([pages, torch.full((B, Hkv, K - n), -1, device=q.device)], -1)
    return pages.to(torch.int32)


def _plain_sparse(s):
    case = s["case"]
    B, H, Hkv, D, p, K = (case[n] for n in ("B", "H", "Hkv", "D", "page", "K"))
    G = H // Hkv
    pages = _plain_select(s)
    lens = s["lens"]
    at = pages.clamp_min(0).long()
    phys = s["table"].long().gather(1, at.flatten(1)).view(B, Hkv, K)
    hk = torch.arange(Hkv, device=lens.device)[None, :, None]
    k = _decoded(s["k"][phys, :, hk], case["kt"], torch.float32).flatten(2, 3)  # [B][Hkv][K * page][D]
    v = _decoded(s["v"][phys, :, hk], case["vt"], torch.float32).flatten(2, 3)
    pos = (at[..., None] * p + torch.arange(p, device=lens.device)).flatten(2)
    there = (pages >= 0).repeat_interleave(p, -1) & (pos < lens[:, None, None])
    q = s["q"].float().view(B, Hkv, G, D)
    x = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    if case["softcap"] > 0:
        x = case["softcap"] * torch.tanh(x / case["softcap"])
    if s["alibi"] is not None:
        x = x + s["alibi"].view(1, Hkv, G, 1) * (pos - (lens[:, None, None] - 1))[:, :, None]
    x = torch.where(there[:, :, None], x, -math.inf)
    top = x.amax(-1, keepdim=True)
    sink = None if s["sinks"] is None else s["sinks"].view(1, Hkv, G, 1)
    if sink is not None:
        top = torch.maximum(top, sink)
    safe = torch.where(top == -math.inf, 0, top)
    e = torch.exp(x - safe)
    total = e.sum(-1, keepdim=True)
    if sink is not None:
        total = total + torch.exp(sink - safe)
    o = torch.matmul(e, torch.where(there[..., None], v, 0)) / torch.where(total > 0, total, 1)
    lse = safe + torch.log(total)
    return {"pages": pages, "O": o.reshape(B, H, D).to(ACT[case["act"]]), "lse": lse.reshape(B, H)}


def _own(s):
    import flash_attention_backward_gb300 as fb
    case = s["case"]
    if case["op"] == "pages":
        got = fb.pages_extend(s["lists"], s["news"], s["T"])
        fb.pages_trim(s["lists"], s["keep"])
        return {**got, "table": s["table"], "lens": s["lens"], "free": s["free"], "num_free": s["num_free"]}
    if case["op"] == "bounds":
        fb.page_bounds(s["cache"], s["bounds"], s["lens"], first=s["first"])
        return {"values": _bound_values(s)}
    if case["op"] == "sparse":
        pages = fb.page_select(s["q"], s["cache"], s["bounds"], s["lens"], case["K"], scale=s["scale"], first=case["first"],
                               last=case["last"], alibi_slopes=s["alibi"])
        got = fb.paged_decode(s["q"], s["cache"], s["lens"], scale=s["scale"], alibi_slopes=s["alibi"], softcap=case["softcap"],
                              sinks=s["sinks"], pages=pages)
        return {"pages": pages, **got}
    style = fb.FA_ROPE_HALVES if case["halves"] else fb.FA_ROPE_PAIRS
    turn = dict(rope=s["rope"], rope_style=style, rope_axes=s["axis"])
    if case["op"] == "store":
        fb.cache_append(s["xk"], s["xv"], s["cache"], s["seq"], s["pos"], k_norm=s["wk"], eps=EPS, rope_pos=s["axes_pos"], **turn)
        return fb.cache_read(s["cache"], s["seq"], s["pos"], dtype=torch.float16)
    if case["op"] == "axes":
        return fb.qk_norm_rope(s["q"], s["k"], s["axes_pos"], wq=s["wq"], wk=s["wk"], eps=EPS, dtype=ACT[case["out"]], **turn)
    return fb.qk_norm_rope_backward(s["gq"], s["gk"], s["q"], s["k"], s["axes_pos"], wq=s["wq"], wk=s["wk"], eps=EPS, **turn)


def _plain_bounds_pass(s):
    _plain_bounds(s)
    return {"values": _bound_values(s)}


def run(state):
    if own:
        return _own(state)
    return {"axes": _plain_axes, "axes_back": _plain_axes_back, "store": _plain_store, "pages": _plain_pages,
            "bounds": _plain_bounds_pass, "sparse": _plain_sparse}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------------
# 64-bit values

def _rotation(s, n_rot, halves):
    """The rotations as complex factors, and the component that each pair's first and second member is."""
    i = torch.arange(n_rot // 2, device=s["axis"].device)
    a = torch.empty((s["axes_pos"].shape[1], n_rot // 2), dtype=torch.float64, device=i.device)
    for axis in range(s["axes_pos"].shape[0]):
        on = s["axis"] == axis
        a[:, on] = s["axes_pos"][axis].double()[:, None] * s["inv_freq"][on][None, :]
    first = i if halves else 2 * i
    second = i + n_rot // 2 if halves else 2 * i + 1
    return torch.polar(torch.ones_like(a), a)[:, None, :], first, second


def _rotate64(x, rot, first, second):
    y = x.clone()
    z = torch.complex(x[..., first], x[..., second]) * rot
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _values64(raw, t):
    """Row bytes to 64-bit values by each format's definition (bytes as integers, no reinterpretation of codes)."""
    if t in ("f32", "f16"):
        return raw.contiguous().view(torch.float32 if t == "f32" else torch.float16).double()
    size = {"q8_0": 34, "q4_0": 18}[t]
    by = raw.reshape(*raw.shape[:-1], raw.shape[-1] // size, size)
    d = by[..., 0:2].contiguous().view(torch.float16).double()
    n = by[..., 2:].to(torch.int16)
    if t == "q8_0":
        code = n - 256 * (n >= 128).to(torch.int16)
    else:
        code = torch.cat([n % 16 - 8, n // 16 - 8], -1)
    return (code.double() * d).flatten(-2)


def _stored64(x, t):
    """What a row of 64-bit values reads as after storage in type t."""
    if t == "f32":
        return x.float().double()
    if t == "f16":
        return x.half().double()
    b = x.reshape(*x.shape[:-1], -1, 32)
    mag = b.abs()
    if t == "q8_0":
        most = mag.max(-1, keepdim=True).values
        d = most / 127.0
        c = torch.sign(b) * torch.floor((127.0 * mag) / most.clamp_min(1e-300) + 0.5)
        c = c.clamp(-127, 127)
    else:
        lead = torch.argmax((mag == mag.max(-1, keepdim=True).values) * torch.arange(32, 0, -1, device=x.device), -1, keepdim=True)
        m = torch.gather(b, -1, lead)
        d = -m / 8.0
        c = torch.floor(b / torch.where(d == 0, torch.ones_like(d), d) + 8.5).clamp(0, 15) - 8.0
        c = torch.where(d == 0, torch.zeros_like(c), c)
    return (c * d.float().half().double()).reshape(x.shape)


def _fl(x):
    """One rounding to f32."""
    return x.float().double()


def _exact_pages(s):
    """The requests one after another, from lists."""
    p, T = s["case"]["page"], s["T"]
    lens, news, keep = s["lens"].tolist(), s["news"].tolist(), s["keep"].tolist()
    table, stack = s["table"].tolist(), s["free"].tolist()
    width, F = len(table[0]), int(s["num_free"])
    starts, first, seq, pos, row = [0], [], [], [], []
    asked, left = 0, F
    for b, (n, m) in enumerate(zip(lens, news)):
        m = m if n >= 0 and m > 0 else 0
        end = starts[-1] + m  # (T is never short here)
        good = m > 0 and n + m <= width * p
        need = -(-(n + m) // p) - -(-n // p) if good else 0
        asked += need
        good = good and (need == 0 or asked <= F)
        first.append(n if good else -1)
        if good:
            for i in range(need):
                left -= 1
                table[b][-(-n // p) + i] = stack[left]
            lens[b] += m
        for i in range(m):
            seq.append(b if good else -1)
            pos.append(n + i if good else -1)
            row.append(table[b][(n + i) // p] * p + (n + i) % p if good else -1)
        starts.append(end)
    for x in (seq, pos, row):
        x += [-1] * (T - len(x))
    for b in reversed(range(len(lens))):  # what was taken last goes back first
        if lens[b] >= 0 and keep[b] >= 0:
            k = min(keep[b], lens[b])
            for j in reversed(range(-(-k // p), -(-lens[b] // p))):
                stack[left], table[b][j] = table[b][j], -1
                left += 1
            lens[b] = k
    return {"seq": seq, "pos": pos, "row": row, "starts": starts, "first": first, "table": table, "lens": lens, "free": stack,
            "num_free": [left]}


def _exact_bounds(s):
    """The bounds of the pages that are to be computed: codes and scales [num_pages] in 64 bits."""
    case = s["case"]
    p, D = case["page"], case["D"]
    lens = s["lens"].tolist()
    first = [0] * len(lens) if s["first"] is None else s["first"].tolist()
    codes, scales = s["codes"].double(), s["scales"].double()
    for b, n in enumerate(lens):
        if n <= 0 or first[b] < 0:
            continue
        f = first[b] // p
        use = s["table"][b, f:-(-n // p)].long()
        k = _values64(s["k"][use], case["kt"])
        k = _fl(k)
        last = n - (f + len(use) - 1) * p  # rows of the last page
        top, low = k.max(1).values, k.min(1).values
        top[-1], low[-1] = k[-1, :last].max(0).values, k[-1, :last].min(0).values
        top, low = (t.reshape(len(use), case["Hkv"], D // 32, 32) for t in (top, low))
        most = torch.maximum(top.abs(), low.abs()).max(-1, keepdim=True).values
        d = _fl(most / 127.0)
        d[most <= _fl(torch.tensor(TINY, dtype=torch.float64))] = 0
        one = torch.where(d > 0, d, torch.ones_like(d))
        up = torch.ceil(_fl(top / one)).clamp(-127, 127) * (d > 0)
        down = torch.floor(_fl(low / one)).clamp(-127, 127) * (d > 0)
        codes[use, :, 0], codes[use, :, 1] = up.flatten(-2), down.flatten(-2)
        scales[use] = d[..., 0]
    return codes, scales


def _exact_select(s, codes, scales, b, n):
    """The pages of sequence b's n positions, for each KV head."""
    case = s["case"]
    H, Hkv, D, p, K = (case[x] for x in ("H", "Hkv", "D", "page", "K"))
    count = -(-n // p)
    use = s["table"][b, :count].long()
    j = torch.arange(count, device=use.device)
    out = []
    for hk in range(Hkv):
        best = torch.full((count,), -math.inf, dtype=torch.float64, device=use.device)
        for h in range(hk * (H // Hkv), (hk + 1) * (H // Hkv)):
            q = s["q"][b, h].double().reshape(-1, 32)
            m = q.abs().max(-1, keepdim=True).values
            zero = m <= 1e-30
            m = torch.where(zero, torch.ones_like(m), m)
            c = torch.round(_fl(q * _fl(127.0 / m))).clamp(-127, 127) * ~zero
            e = _fl(m / 127.0) * ~zero
            hi, lo = (codes[use, hk, i].reshape(count, -1, 32) for i in (0, 1))
            term = torch.maximum(hi * c, lo * c).sum(-1)  # whole numbers
            term = _fl(_fl(term * scales[use, hk]) * e[:, 0])
            while term.shape[-1] > 1:
                term = _fl(term[:, ::2] + term[:, 1::2])
            x = _fl(term[:, 0] * torch.tensor(s["scale"], dtype=torch.float32).double())
            if s["alibi"] is not None:
                x = _fl(x + _fl(s["alibi"][h].double() * (torch.clamp((j + 1) * p, max=n) - n)))
            best = torch.maximum(best, x)
        best[:case["first"]] = math.inf
        if case["last"]:
            best[max(0, count - case["last"]):] = math.inf
        take = torch.sort(best, descending=True, stable=True).indices[:K]
        out.append(torch.sort(take).values)
    return out


def _exact_sparse(s):
    case = s["case"]
    B, H, Hkv, D, p, K = (case[x] for x in ("B", "H", "Hkv", "D", "page", "K"))
    G = H // Hkv
    codes, scales = _exact_bounds(s)
    pages = torch.full((B, Hkv, K), -1, dtype=torch.int32, device="cuda")
    O = torch.zeros((B, H, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, H), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lens(case)):
        chosen = _exact_select(s, codes, scales, b, n) if n else [None] * Hkv
        for hk in range(Hkv):
            if n:
                take = chosen[hk]
                pages[b, hk, :len(take)] = take.int()
                pos = (take[:, None] * p + torch.arange(p, device=take.device)).flatten()
                use = s["table"][b, take].long()
                k = _values64(s["k"][use, :, hk].flatten(0, 1), case["kt"])[pos < n]
                v = _values64(s["v"][use, :, hk].flatten(0, 1), case["vt"])[pos < n]
                pos = pos[pos < n]
            for h in range(hk * G, (hk + 1) * G):
                every = torch.empty(0, dtype=torch.float64, device="cuda")
                if n:
                    x = (k @ s["q"][b, h].double()) * s["scale"]
                    if case["softcap"] > 0:
                        x = case["softcap"] * torch.tanh(x / case["softcap"])
                    if s["alibi"] is not None:
                        x = x + s["alibi"][h].double() * (pos.double() - (n - 1))
                    every = x
                if s["sinks"] is not None:
                    every = torch.cat([every, s["sinks"][h:h + 1].double()])
                if every.numel():
                    lse[b, h] = torch.logsumexp(every, 0)
                if n:
                    O[b, h] = torch.exp(x - lse[b, h]) @ v
    return {"pages": pages, "O": O, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "pages":
        return {n: torch.tensor(x, dtype=torch.int32) for n, x in _exact_pages(s).items()}
    D = case["D"]
    if case["op"] == "bounds":
        codes, scales = _exact_bounds(s)
        return {"values": codes.reshape(*codes.shape[:3], -1, 32) * scales[:, :, None, :, None]}
    if case["op"] == "sparse":
        return _exact_sparse(s)
    n_rot = 2 * s["axis"].numel()
    rot = _rotation(s, n_rot, case["halves"])
    if case["op"] == "store":
        k = s["xk"].double()
        if s["wk"] is not None:
            k = k / torch.sqrt(k.pow(2).sum(-1, keepdim=True) / D + EPS) * s["wk"].double()
        k = _rotate64(k, *rot)
        return {"k": _stored64(k, case["kt"]), "v": _stored64(s["xv"].double(), case["vt"])}
    out = {}
    for n in ("q", "k"):
        x, w = s[n].double(), s["w" + n].double()
        rms = torch.sqrt(x.pow(2).sum(-1, keepdim=True) / D + EPS)
        unit = x / rms
        if case["op"] == "axes":
            out[n] = _rotate64(unit * w, *rot)
        else:
            g = _rotate64(s["g" + n].double(), rot[0].conj(), rot[1], rot[2])
            out["dw" + n] = torch.einsum("nhd,nhd->d", g, unit)
            h = g * w
            out["d" + n] = (h - unit * (h * unit).sum(-1, keepdim=True) / D) / rms
    return out
