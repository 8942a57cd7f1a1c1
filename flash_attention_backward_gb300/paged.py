"""PyTorch-facing wrappers of fa_paged.h: the paged raw cache, and the per-head norm and rotation.

Each call allocates its outputs and workspace with PyTorch and enqueues on the current stream of the
tensors' device (or on `stream`).  No autograd graph is recorded: qk_norm_rope_backward() is called as
backward() is.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
from typing import Optional

import torch

from . import _native as nat
from ._fast_path import fast_path
from .api import FaBackError, Workspace, _check, _ptr


def _load_fast():
    """The plain form of the calls below, in C++ (csrc/py_fast.cpp), or None where it is not built for this
    PyTorch and interpreter: the same calls are then made from here, at a few microseconds more each."""
    path = fast_path()
    if path is None or not os.path.exists(path):
        return None
    try:
        spec = importlib.util.spec_from_file_location(__package__ + "._fast", path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        return module
    except ImportError:
        return None


_fast = _load_fast()


def look_for_fast() -> None:
    """Take the marshalling module that has been built since this one was imported; the one that it has stays."""
    global _fast
    if _fast is None:
        _fast = _load_fast()


_ACT = {torch.float32: nat.FA_ACT_F32, torch.float16: nat.FA_ACT_F16, torch.bfloat16: nat.FA_ACT_BF16}
_F32, _I32, _empty = torch.float32, torch.int32, torch.empty


def _bind():
    """Hand the library's entry points to _fast, once; False without it."""
    global _plain
    if _fast is None:
        return False
    L = nat.lib()
    _fast.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
        L.fa_qk_norm_rope, L.fa_qk_norm_rope_backward, L.fa_qk_norm_rope_backward_workspace_size, L.fa_cache_append,
        L.fa_cache_read, L.fa_paged_decode, L.fa_paged_decode_workspace_size)))
    _plain = True
    return True


_plain = False  # _fast is bound

# These calls are made once a layer and step, on small tensors, so what they cost on the host counts:
# each argument is looked at once, and what a refusal says is put together only when there is one.


def _act(t: torch.dtype) -> int:
    act = _ACT.get(t)
    if act is None:
        raise FaBackError(f"activations are float32, float16 or bfloat16, not {t}")
    return act


def _expect(name: str, t: torch.Tensor, dtype, shape, device) -> int:
    """The address of t, which is contiguous, of this type, shape (a tuple) and device."""
    if t is None:
        raise FaBackError(f"{name}: contiguous {dtype} {tuple(shape)} on {device} expected, got None")
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return t.data_ptr()
    raise FaBackError(f"{name}: contiguous {dtype} {tuple(shape)} on {device} expected, got {t.dtype} "
                      f"{tuple(t.shape)}, strides {t.stride()}, on {t.device}")


def _count(name: str, t: torch.Tensor) -> int:
    """The tokens of t [T]..."""
    if t.dim() == 0:
        raise FaBackError(f"{name}: a tensor of tokens expected, got one value")
    return t.shape[0]


def _heads(name: str, t: torch.Tensor, N: int, D: int, dtype, device):
    """Heads and strides (token, head) of t [N][heads][D], possibly a view whose components are contiguous."""
    if t.dim() == 3 and t.dtype is dtype and t.device == device:
        n, heads, d = t.shape
        row, head, comp = t.stride()
        if n == N < 2 ** 31 and d == D and ((comp == 1 and row >= 0 and head >= 0) or not t.numel()):
            return heads, row, head
    raise FaBackError(f"{name}: {dtype} [{N}][heads][{D}] with contiguous components on {device} expected, got "
                      f"{t.dtype} {tuple(t.shape)}, strides {t.stride()}, on {t.device}")


class _On:
    """Around a call: its stream's device is current, and with `stream` given, what it allocates belongs
    to that stream.  Only made where that is not so already."""

    def __init__(self, device: torch.device, stream: Optional[torch.cuda.Stream]):
        self._guard = torch.cuda.device(device) if stream is None else torch.cuda.stream(stream)

    def __enter__(self):
        self._guard.__enter__()

    def __exit__(self, *exc):
        self._guard.__exit__(*exc)


def _index(device: torch.device) -> int:
    if device.type != "cuda":
        raise FaBackError(f"CUDA tensors expected, got {device}")
    return device.index


def _call(fn, device: torch.device, stream: Optional[torch.cuda.Stream]):
    """fn(stream handle) on the current stream of the device, or on `stream`."""
    index = _index(device)
    if stream is not None and stream.device != device:
        raise FaBackError(f"stream: one of {device} expected, where the tensors are, got one of {stream.device}")
    if stream is None and index == torch._C._cuda_getDevice():
        return fn(torch._C._cuda_getCurrentRawStream(index))
    with _On(device, stream):
        return fn(torch.cuda.current_stream(device).cuda_stream if stream is None else stream.cuda_stream)


def rope_frequencies(n_rot: int, base: float = 10000.0, *, scale: float = 1.0, factors=None,
                     device="cuda") -> torch.Tensor:
    """The frequencies scale * base^(-2 i / n_rot) / factors[i] as the rotation takes them: int64
    [n_rot / 2], turns per position in units of 2^-64 (fa_rope of the header).  Made once and kept."""
    out = torch.empty(max(n_rot, 0) // 2, dtype=torch.int64)
    if factors is not None:
        factors = torch.as_tensor(factors, dtype=torch.float32, device="cpu").contiguous()
        if factors.shape != out.shape:
            raise FaBackError(f"factors: {out.numel()} values expected")
    _check(nat.fa_rope_frequencies(n_rot, base, scale, _ptr(factors), out.data_ptr()))
    return out.to(device)


def _rope(rope: Optional[torch.Tensor], style: int, device) -> Optional[nat.fa_rope]:
    if rope is None:
        return None
    if rope.dtype is not torch.int64 or rope.dim() != 1 or rope.device != device or not rope.is_contiguous():
        raise FaBackError("rope: the contiguous int64 frequencies of rope_frequencies() on the tensors' device expected")
    return nat.fa_rope(rope.data_ptr(), 2 * rope.numel(), style)


class PagedCache:
    """A paged raw K/V cache: pools k and v (uint8 [num_pages][page_size][Hkv][row]) of cache types k_type
    and v_type, and page_table (int32 [B][max_pages]).  Holds the tensors; nothing is copied, so pools and
    table may be edited in place between calls.  It is of the tensors that it was made with: for others (a pool
    that has grown) make another one."""

    def __init__(self, k: torch.Tensor, k_type: int, v: torch.Tensor, v_type: int, page_table: torch.Tensor, *, D: int,
                 Dv: int):
        self.k, self.v, self.page_table = k, v, page_table
        self.k_type, self.v_type, self.D, self.Dv = k_type, v_type, D, Dv
        if k.dim() != 4 or v.dim() != 4:
            raise FaBackError("pools: uint8 [num_pages][page_size][Hkv][row] expected")
        self.num_pages, self.page_size, self.Hkv = k.shape[:3]
        lead = tuple(k.shape[:3])
        _expect("k", k, torch.uint8, lead + (nat.fa_row_bytes(k_type, D),), k.device)
        _expect("v", v, torch.uint8, lead + (nat.fa_row_bytes(v_type, Dv),), k.device)
        if page_table.dim() != 2:
            raise FaBackError("page_table: int32 [B][max_pages] expected")
        _expect("page_table", page_table, torch.int32, tuple(page_table.shape), k.device)
        self.B, self.max_pages = page_table.shape
        self.device = k.device
        self.c = nat.fa_paged_cache(k.data_ptr(), v.data_ptr(), page_table.data_ptr(), k_type, v_type, self.num_pages,
                                    self.page_size, self.B, self.max_pages, self.Hkv, D, Dv)
        self._at, self._index = ctypes.addressof(self.c), self.device.index
        self._ws = {}  # decode workspace bytes by query head count

    def __setattr__(self, name, value):
        if name in self.__dict__:  # the kernels would go on with the old tensor's address
            raise FaBackError(f"{name}: a PagedCache keeps what it was made with; make another one")
        super().__setattr__(name, value)

    def decode_workspace_size(self, H: int) -> int:
        """fa_paged_decode_workspace_size() of this cache (0: the arguments are invalid)."""
        n = self._ws.get(H)
        if n is None:
            with torch.cuda.device(self.device):
                n = self._ws[H] = nat.fa_paged_decode_workspace_size(self.c, H)
        return n


def cache_append(k: torch.Tensor, v: torch.Tensor, cache: PagedCache, seq: torch.Tensor, pos: torch.Tensor, *,
                 k_norm: Optional[torch.Tensor] = None, eps: float = 1e-6, rope: Optional[torch.Tensor] = None,
                 rope_style: int = nat.FA_ROPE_HALVES, stream: Optional[torch.cuda.Stream] = None) -> None:
    """Store keys k [T][Hkv][D] and values v [T][Hkv][Dv] (f32, f16 or bf16; may be views) as positions
    pos [T] of sequences seq [T] (int32; negative: a padding token, skipped) of the cache, quantised to
    its types.  Keys are normalised by k_norm (f32 [D], or None) and rotated by pos with the
    frequencies rope (rope_frequencies(), or None) on the way."""
    if stream is None and cache._index is not None and (_plain or _bind()) and _fast.append(
            k, v, cache._at, cache._index, seq, pos, k_norm, eps, rope, rope_style):
        return
    dev, T = cache.device, _count("k", k)
    act = _act(k.dtype)
    hk, k_row, k_head = _heads("k", k, T, cache.D, k.dtype, dev)
    hv, v_row, v_head = _heads("v", v, T, cache.Dv, k.dtype, dev)
    if hk != cache.Hkv or hv != hk:
        raise FaBackError(f"k, v: {cache.Hkv} heads expected")
    p_seq = _expect("seq", seq, _I32, (T,), dev)
    p_pos = _expect("pos", pos, _I32, (T,), dev)
    p_norm = None if k_norm is None else _expect("k_norm", k_norm, _F32, (cache.D,), dev)
    r = _rope(rope, rope_style, dev)
    views = nat.fa_kv_views(k_row, k_head, v_row, v_head)
    _check(_call(lambda s: nat.fa_cache_append(k.data_ptr(), v.data_ptr(), act, views, cache.c, p_seq, p_pos, T, p_norm,
                                               eps, r, s), dev, stream))


def cache_read(cache: PagedCache, seq: torch.Tensor, pos: torch.Tensor, *, dtype=torch.float32,
               out: Optional[dict] = None, stream: Optional[torch.cuda.Stream] = None) -> dict:
    """The cache's rows at positions pos [T] of sequences seq [T]: {"k": [T][Hkv][D], "v": [T][Hkv][Dv]} of
    dtype, or with dtype=torch.uint8 the raw rows [T][Hkv][row], the contiguous cache that backward()
    and forward() take.  Rows of skipped tokens (negative seq or pos) are not written."""
    if stream is None and out is None and cache._index is not None and (_plain or _bind()):
        got = _fast.read(cache._at, cache._index, seq, pos, dtype)
        if got is not None:
            return got
    dev, T = cache.device, _count("seq", seq)
    if dtype is torch.uint8:
        act, nk, nv = nat.FA_ACT_RAW, cache.k.shape[3], cache.v.shape[3]
    else:
        act, nk, nv = _act(dtype), cache.D, cache.Dv
    p_seq = _expect("seq", seq, _I32, (T,), dev)
    p_pos = _expect("pos", pos, _I32, (T,), dev)

    def run(s):
        o = out
        if o is None:
            o = {"k": _empty((T, cache.Hkv, nk), dtype=dtype, device=dev), "v": _empty((T, cache.Hkv, nv), dtype=dtype, device=dev)}
            p_k, p_v = o["k"].data_ptr(), o["v"].data_ptr()
        else:
            p_k = _expect("out k", o["k"], dtype, (T, cache.Hkv, nk), dev)
            p_v = _expect("out v", o["v"], dtype, (T, cache.Hkv, nv), dev)
        _check(nat.fa_cache_read(cache.c, p_seq, p_pos, T, act, p_k, p_v, s))
        return o

    return _call(run, dev, stream)


def paged_decode(q: torch.Tensor, cache: PagedCache, seq_lens: torch.Tensor, *, scale: float,
                 alibi_slopes: Optional[torch.Tensor] = None, softcap: float = 0.0,
                 sinks: Optional[torch.Tensor] = None, out: Optional[dict] = None,
                 workspace: Optional[Workspace] = None, stream: Optional[torch.cuda.Stream] = None) -> dict:
    """Attention of one new token per sequence: q [B][H][D] (f32, f16 or bf16; may be a view) over the first
    seq_lens [B] (int32) positions of the cache's sequences: {"O": [B][H][Dv] of q's type, "lse": [B][H] f32}.
    ALiBi slopes and sinks (f32 [H]) and the soft cap are those of backward().  A negative length marks a
    padding slot, whose rows are not written."""
    if stream is None and out is None and workspace is None and cache._index is not None and (_plain or _bind()):
        got = _fast.decode(q, cache._at, cache._index, seq_lens, scale, alibi_slopes, softcap, sinks)
        if got is not None:
            return got
    dev, B, dtype = cache.device, cache.B, q.dtype
    act = _act(dtype)
    H, q_row, q_head = _heads("q", q, B, cache.D, dtype, dev)
    p_len = _expect("seq_lens", seq_lens, _I32, (B,), dev)
    p_alibi = None if alibi_slopes is None else _expect("alibi_slopes", alibi_slopes, _F32, (H,), dev)
    p_sinks = None if sinks is None else _expect("sinks", sinks, _F32, (H,), dev)
    _index(dev)

    def run(s):
        o = out
        need = cache._ws.get(H) or cache.decode_workspace_size(H)
        if o is None:
            o = {"O": _empty((B, H, cache.Dv), dtype=dtype, device=dev), "lse": _empty((B, H), dtype=_F32, device=dev)}
            p_o, p_lse = o["O"].data_ptr(), o["lse"].data_ptr()
        else:
            p_o = _expect("out O", o["O"], dtype, (B, H, cache.Dv), dev)
            p_lse = _expect("out lse", o["lse"], _F32, (B, H), dev)
        ws = _empty((need,), dtype=torch.uint8, device=dev) if workspace is None else workspace.get(need)
        _check(nat.fa_paged_decode(q.data_ptr(), act, q_row, q_head, cache.c, p_len, H, scale, p_alibi, softcap, p_sinks,
                                   p_o, p_lse, ws.data_ptr(), need, s))
        return o

    return _call(run, dev, stream)


def _qk(q, k):
    """Shape, device, dtype of q and the head counts and views of q and k (k may be None)."""
    if q.dim() != 3:
        raise FaBackError(f"q: [N][H][D] expected, got {tuple(q.shape)}")
    (N, H, D), dev, dtype = q.shape, q.device, q.dtype
    _, q_row, q_head = _heads("q", q, N, D, dtype, dev)
    Hkv, k_row, k_head = (0, 0, 0) if k is None else _heads("k", k, N, D, dtype, dev)
    return N, H, D, dev, dtype, Hkv, nat.fa_qk_views(q_row, q_head, k_row, k_head)


def qk_norm_rope(q: torch.Tensor, k: Optional[torch.Tensor], pos: Optional[torch.Tensor], *,
                 wq: Optional[torch.Tensor] = None, wk: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 rope: Optional[torch.Tensor] = None, rope_style: int = nat.FA_ROPE_HALVES, dtype=None,
                 out: Optional[dict] = None, stream: Optional[torch.cuda.Stream] = None) -> dict:
    """RMS norm of every head (weights wq, wk f32 [D]; None: not normalised) and rotation by pos [N]
    (int32) of queries q [N][H][D] and keys k [N][Hkv][D] (f32, f16 or bf16, possibly views of one
    projection; k may be None): {"q", "k"}, contiguous, of dtype (default q's)."""
    if stream is None and out is None and (_plain or _bind()):
        got = _fast.norm(q, k, pos, wq, wk, eps, rope, rope_style, dtype)
        if got is not None:
            return got
    N, H, D, dev, x_dtype, Hkv, views = _qk(q, k)
    dtype = x_dtype if dtype is None else dtype
    x_type, y_type = _act(x_dtype), _act(dtype)
    p_wq = None if wq is None else _expect("wq", wq, _F32, (D,), dev)
    p_wk = None if wk is None else _expect("wk", wk, _F32, (D,), dev)
    r = _rope(rope, rope_style, dev)
    p_pos = None if r is None else _expect("pos", pos, _I32, (N,), dev)

    def run(s):
        o = out
        if o is None:
            o = {"q": _empty((N, H, D), dtype=dtype, device=dev), "k": None if k is None else _empty((N, Hkv, D), dtype=dtype, device=dev)}
            p_q, p_k = o["q"].data_ptr(), None if k is None else o["k"].data_ptr()
        else:
            p_q = _expect("out q", o["q"], dtype, (N, H, D), dev)
            p_k = None if k is None else _expect("out k", o["k"], dtype, (N, Hkv, D), dev)
        _check(nat.fa_qk_norm_rope(q.data_ptr(), _ptr(k), x_type, views, p_wq, p_wk, eps, p_pos, r, N, H, Hkv, D, p_q, p_k,
                                   y_type, s))
        return o

    return _call(run, dev, stream)


def qk_norm_rope_backward(gq: torch.Tensor, gk: Optional[torch.Tensor], q: torch.Tensor, k: Optional[torch.Tensor],
                          pos: Optional[torch.Tensor], *, wq: Optional[torch.Tensor] = None,
                          wk: Optional[torch.Tensor] = None, eps: float = 1e-6, rope: Optional[torch.Tensor] = None,
                          rope_style: int = nat.FA_ROPE_HALVES, out: Optional[dict] = None,
                          workspace: Optional[Workspace] = None,
                          stream: Optional[torch.cuda.Stream] = None) -> dict:
    """The gradient of qk_norm_rope(): given gq [N][H][D] and gk [N][Hkv][D] (contiguous, e.g. backward()'s dQ
    and dK) and the forward's inputs, {"dq", "dk" of q's type, "dwq", "dwk" f32 [D] (with the weights)}."""
    if stream is None and out is None and workspace is None and (_plain or _bind()):
        got = _fast.norm_back(gq, gk, q, k, pos, wq, wk, eps, rope, rope_style)
        if got is not None:
            return got
    N, H, D, dev, dtype, Hkv, views = _qk(q, k)
    if (gk is None) != (k is None):
        raise FaBackError("gk and k are given together")
    x_type, y_type = _act(dtype), _act(gq.dtype)
    p_gq = _expect("gq", gq, gq.dtype, (N, H, D), dev)
    p_gk = None if gk is None else _expect("gk", gk, gq.dtype, (N, Hkv, D), dev)
    p_wq = None if wq is None else _expect("wq", wq, _F32, (D,), dev)
    p_wk = None if wk is None else _expect("wk", wk, _F32, (D,), dev)
    r = _rope(rope, rope_style, dev)
    p_pos = None if r is None else _expect("pos", pos, _I32, (N,), dev)

    def run(s):
        o = out
        if o is None:
            o = {"dq": _empty((N, H, D), dtype=dtype, device=dev)}
            if k is not None:
                o["dk"] = _empty((N, Hkv, D), dtype=dtype, device=dev)
            if wq is not None:
                o["dwq"] = _empty((D,), dtype=_F32, device=dev)
            if wk is not None and k is not None:
                o["dwk"] = _empty((D,), dtype=_F32, device=dev)
        else:
            for name, t, shape in (("dq", dtype, (N, H, D)), ("dk", dtype, (N, Hkv, D)), ("dwq", _F32, (D,)), ("dwk", _F32, (D,))):
                if o.get(name) is not None:
                    _expect("out " + name, o[name], t, shape, dev)
        need = nat.fa_qk_norm_rope_backward_workspace_size(N, H, Hkv, D)
        ws = _empty((need,), dtype=torch.uint8, device=dev) if workspace is None else workspace.get(need)
        _check(nat.fa_qk_norm_rope_backward(
            p_gq, p_gk, y_type, q.data_ptr(), _ptr(k), x_type, views, p_wq, p_wk, eps, p_pos, r, N, H, Hkv, D,
            o["dq"].data_ptr(), _ptr(o.get("dk")), _ptr(o.get("dwq")), _ptr(o.get("dwk")), ws.data_ptr(), need, s))
        return o

    return _call(run, dev, stream)
