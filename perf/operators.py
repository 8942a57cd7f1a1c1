"""The paged-cache and per-head operators: their cases, plain forms and 64-bit values.

Operators
  decode    one new token per sequence attends over a paged raw K/V cache (paged_decode)
  append    K and V of T tokens are normalised (K), rotated (K) and stored into a paged raw cache in
            the cache's own types (cache_append); the rows are then read back decoded (cache_read)
  norm      RMS norm of every query and key head and the position rotation (qk_norm_rope)
  norm_back the gradient of that with respect to q, k and both norm weights (qk_norm_rope_backward)

Cache rows: f32 and f16 values; q8_0 blocks of 32 (binary16 scale d, 32 int8 codes, value code * d);
q4_0 blocks of 32 (binary16 scale d, 16 bytes, byte b holding element b low and b + 16 high, value
(nibble - 8) * d).  A pool is [num_pages][page_size][Hkv][row bytes]; position j of sequence b is row
j % page_size of page page_table[b][j // page_size].  Rotation angle of pair i at position p: p * inv_freq[i].
"""
import math

import torch

own = False

ROW = {"f32": lambda D: 4 * D, "f16": lambda D: 2 * D, "q8_0": lambda D: D // 32 * 34, "q4_0": lambda D: D // 32 * 18}
CODE = {"f32": 0, "f16": 1, "q8_0": 2, "q4_0": 3}
ACT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ACT_BYTES = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-6


# ------------------------------------------------------------------------------------------------
# cases

def _decode(name, B, max_len, lens, H, Hkv, D, kt, vt, act, page, softcap=0.0, alibi=False, sinks=False):
    return {"name": name, "op": "decode", "B": B, "max_len": max_len, "lens": lens, "H": H, "Hkv": Hkv, "D": D, "kt": kt,
            "vt": vt, "act": act, "page": page, "softcap": softcap, "alibi": alibi, "sinks": sinks}


def _append(name, T, B, start, Hkv, D, kt, vt, act, page, n_rot, halves, k_norm):
    return {"name": name, "op": "append", "T": T, "B": B, "start": start, "Hkv": Hkv, "D": D, "kt": kt, "vt": vt,
            "act": act, "page": page, "n_rot": n_rot, "halves": halves, "k_norm": k_norm}


def _norm(name, op, N, H, Hkv, D, act, out, n_rot, halves, fused, start):
    return {"name": name, "op": op, "N": N, "H": H, "Hkv": Hkv, "D": D, "act": act, "out": out, "n_rot": n_rot,
            "halves": halves, "fused": fused, "start": start}


def listed():
    return [
        # one sequence with a short cache, as in an interactive session: the call's latency
        _decode("decode_short_q8", 1, 512, "full", 8, 2, 128, "q8_0", "q8_0", "f32", 64),
        # one sequence at the long-context length of the benchmark
        _decode("decode_long_q8", 1, 75520, "full", 24, 4, 256, "q8_0", "q8_0", "f32", 64),
        # a serving batch of unequal lengths, some slots empty, binary16 cache, small pages
        _decode("decode_batch_f16", 48, 8192, "ragged", 32, 8, 128, "f16", "f16", "bf16", 16),
        # mixed cache types with every score extension; the page is no multiple of a tile
        _decode("decode_mixed_ext", 24, 6000, "ragged", 24, 4, 256, "q4_0", "q8_0", "f16", 40, 30.0, True, True),
        # a decode step's new rows: one token for each of 64 sequences
        _append("append_step_q8", 64, 64, 4000, 4, 256, "q8_0", "q8_0", "f32", 64, 256, True, True),
        # a prompt of one sequence going into a quantised cache
        _append("append_prompt_q8", 2048, 1, 73000, 4, 256, "q8_0", "q8_0", "f32", 64, 256, True, True),
        # prompts of several sequences in one call, mixed types, rotation of a part of each head in neighbouring pairs
        _append("append_ragged_mixed", 5003, 7, 11, 8, 128, "f16", "q4_0", "bf16", 16, 64, False, False),
        # a decode step's queries and keys
        _norm("norm_step_bf16", "norm", 64, 32, 8, 128, "bf16", "bf16", 128, True, True, 9000),
        # the queries and keys of the long-context shape's step, in the f32 that the attention takes
        _norm("norm_long_f32", "norm", 2048, 24, 4, 256, "f32", "f32", 256, True, False, 73472),
        # a long prompt read out of one fused projection
        _norm("norm_prompt_bf16", "norm", 16411, 8, 2, 64, "bf16", "f32", 32, False, True, 0),
        # training: the long-context shape's dQ and dK going back
        _norm("norm_back_f32", "norm_back", 2048, 24, 4, 256, "f32", "f32", 256, True, False, 73472),
        # training in 16-bit activations with an odd token count
        _norm("norm_back_bf16", "norm_back", 8191, 32, 8, 128, "bf16", "bf16", 128, True, True, 0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "append", "norm", "norm_back"])
    D = rng.choice([64, 128, 256])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    types = ["f32", "f16", "q8_0", "q4_0"]
    if op == "decode":
        G = rng.choice([1, 2, 3, 4, 6, 8, 12])
        kt, vt = rng.choice(types), rng.choice(types)
        B = _log(rng, 1, 96)
        top = int(200e6 / (B * Hkv * (ROW[kt](D) + ROW[vt](D))))  # bytes of the cache that is read
        return _decode("", B, _log(rng, 1, max(1, min(100000, top))), rng.choice(["full", "ragged"]), G * Hkv, Hkv, D, kt, vt,
                       rng.choice(["f32", "f16", "bf16"]), rng.choice([16, 32, 48, 64, 128, 256]),
                       rng.choice([0.0, 0.0, 30.0, 50.0]), rng.random() < 0.3, rng.random() < 0.3)
    halves = rng.random() < 0.6
    n_rot = rng.choice([D, D // 2, D // 4])
    act = rng.choice(["f32", "f16", "bf16"])
    if op == "append":
        T = _log(rng, 1, min(8192, 12000000 // (Hkv * D)))
        return _append("", T, min(T, _log(rng, 1, 64)), rng.randrange(0, 100000), Hkv, D, rng.choice(types), rng.choice(types),
                       act, rng.choice([16, 32, 48, 64, 128]), n_rot, halves, rng.random() < 0.6)
    H = Hkv * rng.choice([1, 2, 3, 4, 6, 8])
    N = _log(rng, 1, min(20000, 30000000 // ((H + Hkv) * D)))
    return _norm("", op, N, H, Hkv, D, act, act if op == "norm_back" else rng.choice([act, "f32"]), n_rot, halves,
                 rng.random() < 0.5, rng.randrange(0, 1000000))


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


def _split(case):
    """(sequence, position) of each appended token: the sequences' shares are unequal."""
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


def work(case):
    D, Hkv, a = case["D"], case["Hkv"], ACT_BYTES[case["act"]]
    if case["op"] == "decode":
        n = sum(_lens(case))
        B, H = case["B"], case["H"]
        return {"bytes": n * Hkv * (ROW[case["kt"]](D) + ROW[case["vt"]](D)) + 2 * B * H * D * a + 4 * B * H, "flops": 4 * H * D * n}
    if case["op"] == "append":
        rows = case["T"] * Hkv
        raw = ROW[case["kt"]](D) + ROW[case["vt"]](D)
        # new rows read and stored; the stored rows read and given out in binary16
        return {"bytes": rows * (2 * D * a + 2 * raw + 2 * D * 2), "flops": rows * D * 12}
    rows = case["N"] * (case["H"] + Hkv)
    o = ACT_BYTES[case["out"]]
    if case["op"] == "norm":
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


def _pages(gen, B, max_pages, dev):
    n = B * max_pages + 3
    return n, torch.randperm(n, generator=gen, device=dev)[: B * max_pages].reshape(B, max_pages).to(torch.int32)


def _pool(gen, n_rows, Hkv, D, t, dev, amp):
    out = torch.empty((n_rows, Hkv, ROW[t](D)), dtype=torch.uint8, device=dev)
    step = max(1, (1 << 25) // (Hkv * D))
    for r in range(0, n_rows, step):
        m = min(step, n_rows - r)
        out[r:r + m] = _quantise(amp * torch.randn((m, Hkv, D), generator=gen, device=dev), t)
    return out


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    D, Hkv = case["D"], case["Hkv"]
    act = ACT[case["act"]]
    s = {"case": case}

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    if case["op"] == "decode":
        B, H, page = case["B"], case["H"], case["page"]
        max_pages = -(-case["max_len"] // page)
        n_pages, s["table"] = _pages(gen, B, max_pages, dev)
        s["k"] = _pool(gen, n_pages * page, Hkv, D, case["kt"], dev, 1.0).view(n_pages, page, Hkv, -1)
        s["v"] = _pool(gen, n_pages * page, Hkv, D, case["vt"], dev, 1.0).view(n_pages, page, Hkv, -1)
        s["lens"] = torch.tensor(_lens(case), dtype=torch.int32, device=dev)
        s["q"] = normal(B, H, D).to(act)
        s["scale"] = D ** -0.5
        s["alibi"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], device=dev) if case["alibi"] else None
        s["sinks"] = 1.0 + normal(H) if case["sinks"] else None
    elif case["op"] == "append":
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
        s["k"] = torch.zeros((n_pages, page, Hkv, ROW[case["kt"]](D)), dtype=torch.uint8, device=dev)
        s["v"] = torch.zeros((n_pages, page, Hkv, ROW[case["vt"]](D)), dtype=torch.uint8, device=dev)
        s["xk"], s["xv"] = normal(T, Hkv, D).to(act), normal(T, Hkv, D).to(act)
        s["wk"] = 1.0 + 0.1 * normal(D) if case["k_norm"] else None
        s["inv_freq"], s["rope"] = _rope(case["n_rot"], 10000.0, dev)
    else:
        N, H = case["N"], case["H"]
        x = normal(N, H + 2 * Hkv, D).to(act) if case["fused"] else None  # one projection of q, k and v
        s["q"] = x[:, :H] if case["fused"] else normal(N, H, D).to(act)
        s["k"] = x[:, H:H + Hkv] if case["fused"] else normal(N, Hkv, D).to(act)
        s["pos"] = torch.arange(case["start"], case["start"] + N, dtype=torch.int32, device=dev)
        s["wq"], s["wk"] = 1.0 + 0.1 * normal(D), 1.0 + 0.1 * normal(D)
        s["inv_freq"], s["rope"] = _rope(case["n_rot"], 1000000.0, dev)
        if case["op"] == "norm_back":
            s["gq"], s["gk"] = normal(N, H, D).to(ACT[case["out"]]), normal(N, Hkv, D).to(ACT[case["out"]])
    if own and case["op"] in ("decode", "append"):
        import flash_attention_backward_gb300 as fb
        s["cache"] = fb.PagedCache(s["k"], CODE[case["kt"]], s["v"], CODE[case["vt"]], s["table"], D=D, Dv=D)
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
    a = s["pos"].to(torch.float64)[:, None, None] * s["inv_freq"]
    return torch.cos(a).to(kind), torch.sin(a).to(kind)


def _normed(x, w):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w


def _plain_decode(s):
    case = s["case"]
    B, H, Hkv, D = case["B"], case["H"], case["Hkv"], case["D"]
    at = s["table"].long()
    k = _decoded(s["k"][at].flatten(1, 2), case["kt"], torch.float32)  # [B, L, Hkv, D]
    v = _decoded(s["v"][at].flatten(1, 2), case["vt"], torch.float32)
    q = s["q"].float().view(B, Hkv, H // Hkv, D)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)) * s["scale"]  # [B, Hkv, G, L]
    if case["softcap"] > 0:
        x = case["softcap"] * torch.tanh(x / case["softcap"])
    j = torch.arange(k.shape[1], device=q.device)
    if s["alibi"] is not None:
        x = x + s["alibi"].view(1, Hkv, -1, 1) * (j - (s["lens"][:, None] - 1)).view(B, 1, 1, -1)
    x = torch.where((j < s["lens"][:, None]).view(B, 1, 1, -1), x, -math.inf)
    top = x.amax(-1, keepdim=True)
    sink = None if s["sinks"] is None else s["sinks"].view(1, Hkv, -1, 1)
    if sink is not None:
        top = torch.maximum(top, sink)
    safe = torch.where(top == -math.inf, 0, top)
    e = torch.exp(x - safe)
    total = e.sum(-1, keepdim=True)
    if sink is not None:
        total = total + torch.exp(sink - safe)
    v = torch.where((j < s["lens"][:, None]).view(B, -1, 1, 1), v, 0)
    o = torch.matmul(e, v.permute(0, 2, 1, 3)) / torch.where(total > 0, total, 1)
    lse = safe + torch.log(total)
    return {"O": o.reshape(B, H, D).to(ACT[case["act"]]), "lse": lse.reshape(B, H)}


def _plain_append(s):
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


def _plain_norm(s):
    case = s["case"]
    cos, sin = _angles(s, torch.float32)
    return {n: _turned(_normed(s[n].float(), s["w" + n]), cos, sin, case["halves"], False).to(ACT[case["out"]]) for n in ("q", "k")}


def _plain_norm_back(s):
    case = s["case"]
    cos, sin = _angles(s, torch.float32)
    out = {}
    for n in ("q", "k"):
        x, w = s[n].float(), s["w" + n]
        g = _turned(s["g" + n].float(), cos, sin, case["halves"], True)
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        out["dw" + n] = (g * x * r).to(torch.float64).sum((0, 1)).float()
        h = g * w
        out["d" + n] = (r * (h - x * (r * r * (h * x).mean(-1, keepdim=True)))).to(ACT[case["act"]])
    return out


def _own(s):
    import flash_attention_backward_gb300 as fb
    case = s["case"]
    if case["op"] == "decode":
        return fb.paged_decode(s["q"], s["cache"], s["lens"], scale=s["scale"], alibi_slopes=s["alibi"], softcap=case["softcap"],
                               sinks=s["sinks"])
    style = fb.FA_ROPE_HALVES if case["halves"] else fb.FA_ROPE_PAIRS
    if case["op"] == "append":
        fb.cache_append(s["xk"], s["xv"], s["cache"], s["seq"], s["pos"], k_norm=s["wk"], eps=EPS, rope=s["rope"], rope_style=style)
        return fb.cache_read(s["cache"], s["seq"], s["pos"], dtype=torch.float16)
    if case["op"] == "norm":
        return fb.qk_norm_rope(s["q"], s["k"], s["pos"], wq=s["wq"], wk=s["wk"], eps=EPS, rope=s["rope"], rope_style=style,
                               dtype=ACT[case["out"]])
    return fb.qk_norm_rope_backward(s["gq"], s["gk"], s["q"], s["k"], s["pos"], wq=s["wq"], wk=s["wk"], eps=EPS, rope=s["rope"],
                                    rope_style=style)


def run(state):
    if own:
        return _own(state)
    return {"decode": _plain_decode, "append": _plain_append, "norm": _plain_norm, "norm_back": _plain_norm_back}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------------
# 64-bit values

def _rotation(s, n_rot, halves, D):
    """The rotations as complex factors, and the component that each pair's first and second member is."""
    i = torch.arange(n_rot // 2, device=s["pos"].device)
    a = s["pos"].to(torch.float64)[:, None] * s["inv_freq"][None, :]
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


def exact(case, seed):
    s = prepare(case, seed)
    D, Hkv = case["D"], case["Hkv"]
    if case["op"] == "decode":
        H, G, page = case["H"], case["H"] // Hkv, case["page"]
        O = torch.zeros((case["B"], H, D), dtype=torch.float64, device="cuda")
        lse = torch.full((case["B"], H), -math.inf, dtype=torch.float64, device="cuda")
        for b, n in enumerate(_lens(case)):
            use = s["table"][b, : -(-n // page)].long()
            k = _values64(s["k"][use].flatten(0, 1)[:n], case["kt"])
            v = _values64(s["v"][use].flatten(0, 1)[:n], case["vt"])
            for h in range(H):
                x = (k[:, h // G] @ s["q"][b, h].double()) * s["scale"]
                if case["softcap"] > 0:
                    x = case["softcap"] * torch.tanh(x / case["softcap"])
                if s["alibi"] is not None:
                    x = x + s["alibi"][h].double() * (torch.arange(n, device=x.device, dtype=torch.float64) - (n - 1))
                every = x if s["sinks"] is None else torch.cat([x, s["sinks"][h:h + 1].double()])
                if every.numel():
                    lse[b, h] = torch.logsumexp(every, 0)
                if n:
                    O[b, h] = torch.exp(x - lse[b, h]) @ v[:, h // G]
        return {"O": O, "lse": lse}
    if case["op"] == "append":
        k = s["xk"].double()
        if s["wk"] is not None:
            k = k / torch.sqrt(k.pow(2).sum(-1, keepdim=True) / D + EPS) * s["wk"].double()
        k = _rotate64(k, *_rotation(s, case["n_rot"], case["halves"], D))
        return {"k": _stored64(k, case["kt"]), "v": _stored64(s["xv"].double(), case["vt"])}
    rot = _rotation(s, case["n_rot"], case["halves"], D)
    out = {}
    for n in ("q", "k"):
        x, w = s[n].double(), s["w" + n].double()
        rms = torch.sqrt(x.pow(2).sum(-1, keepdim=True) / D + EPS)
        unit = x / rms
        if case["op"] == "norm":
            out[n] = _rotate64(unit * w, *rot)
        else:
            g = _rotate64(s["g" + n].double(), rot[0].conj(), rot[1], rot[2])
            out["dw" + n] = torch.einsum("nhd,nhd->d", g, unit)
            h = g * w
            out["d" + n] = (h - unit * (h * unit).sum(-1, keepdim=True) / D) / rms
    return out
