"""PyTorch-facing wrappers of fa_paged.h: the paged raw cache, and the per-head norm and rotation.

Each call allocates its outputs and workspace with PyTorch and enqueues on the current stream of the
tensors' device (or on `stream`).
"""
from __future__ import annotations

from typing import Optional

import torch

from . import _native as nat
from .api import FaBackError, Workspace, _check, _ptr

_ACT = {torch.float32: nat.FA_ACT_F32, torch.float16: nat.FA_ACT_F16, torch.bfloat16: nat.FA_ACT_BF16}


def _act(t: torch.dtype) -> int:
    try:
        return _ACT[t]
    except KeyError:
        raise FaBackError(f"activations are float32, float16 or bfloat16, not {t}") from None


def _expect(name: str, t: Optional[torch.Tensor], dtype, shape, device) -> None:
    """t (or None) is contiguous, of this type, shape and device."""
    if t is None:
        return
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or t.device != device or not t.is_contiguous():
        raise FaBackError(f"{name}: contiguous {dtype} {tuple(shape)} on {device} expected, got {t.dtype} "
                          f"{tuple(t.shape)} on {t.device}")


def _heads(name: str, t: torch.Tensor, N: int, D: int, dtype, device) -> torch.Tensor:
    """t [N][heads][D], possibly a view whose components are contiguous."""
    if t.dim() != 3 or t.shape[0] != N or t.shape[2] != D or t.dtype != dtype or t.device != device:
        raise FaBackError(f"{name}: {dtype} [{N}][heads][{D}] on {device} expected, got {t.dtype} {tuple(t.shape)} on "
                          f"{t.device}")
    if t.numel() and (t.stride(2) != 1 or t.stride(0) < 0 or t.stride(1) < 0):
        raise FaBackError(f"{name}: components must be contiguous")
    return t


class _On:
    """The stream that a call enqueues on, with the tensors' device current.  With `stream` given, what
    the call allocates belongs to that stream."""

    def __init__(self, device: torch.device, stream: Optional[torch.cuda.Stream]):
        if device.type != "cuda":
            raise FaBackError(f"CUDA tensors expected, got {device}")
        if stream is not None:
            self._guard = torch.cuda.stream(stream)
        elif device.index != torch.cuda.current_device():
            self._guard = torch.cuda.device(device)
        else:
            self._guard = None
        self.handle = (torch.cuda.current_stream(device) if stream is None else stream).cuda_stream

    def __enter__(self):
        if self._guard is not None:
            self._guard.__enter__()
        return self

    def __exit__(self, *exc):
        if self._guard is not None:
            self._guard.__exit__(*exc)


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


def _rope(rope: Optional[torch.Tensor], style: int, pos: torch.Tensor, N: int, device) -> Optional[nat.fa_rope]:
    if rope is None:
        return None
    if rope.dtype != torch.int64 or rope.dim() != 1 or rope.device != device or not rope.is_contiguous():
        raise FaBackError("rope: the contiguous int64 frequencies of rope_frequencies() on the tensors' device expected")
    _expect("pos", pos, torch.int32, (N,), device)
    return nat.fa_rope(rope.data_ptr(), 2 * rope.numel(), style)


class PagedCache:
    """A paged raw K/V cache: pools k and v (uint8 [num_pages][page_size][Hkv][row]) of cache types k_type
    and v_type, and page_table (int32 [B][max_pages]).  Holds the tensors; nothing is copied, so the
    table may be edited in place between calls."""

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
        self._ws = {}  # decode workspace bytes by query head count

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
    dev, T = cache.device, k.shape[0]
    act = _act(k.dtype)
    _heads("k", k, T, cache.D, k.dtype, dev)
    _heads("v", v, T, cache.Dv, k.dtype, dev)
    if k.shape[1] != cache.Hkv or v.shape[1] != cache.Hkv:
        raise FaBackError(f"k, v: {cache.Hkv} heads expected")
    _expect("seq", seq, torch.int32, (T,), dev)
    _expect("pos", pos, torch.int32, (T,), dev)
    _expect("k_norm", k_norm, torch.float32, (cache.D,), dev)
    r = _rope(rope, rope_style, pos, T, dev)
    views = nat.fa_kv_views(k.stride(0), k.stride(1), v.stride(0), v.stride(1))
    with _On(dev, stream) as on:
        _check(nat.fa_cache_append(k.data_ptr(), v.data_ptr(), act, views, cache.c, seq.data_ptr(), pos.data_ptr(), T,
                                   _ptr(k_norm), eps, r, on.handle))


def cache_read(cache: PagedCache, seq: torch.Tensor, pos: torch.Tensor, *, dtype=torch.float32,
               out: Optional[dict] = None, stream: Optional[torch.cuda.Stream] = None) -> dict:
    """The cache's rows at positions pos [T] of sequences seq [T]: {"k": [T][Hkv][D], "v": [T][Hkv][Dv]} of
    dtype, or with dtype=torch.uint8 the raw rows [T][Hkv][row], the contiguous cache that backward()
    and forward() take.  Rows of skipped tokens (negative seq or pos) are not written."""
    dev, T = cache.device, seq.shape[0]
    raw = dtype == torch.uint8
    act = nat.FA_ACT_RAW if raw else _act(dtype)
    _expect("seq", seq, torch.int32, (T,), dev)
    _expect("pos", pos, torch.int32, (T,), dev)
    nk, nv = (cache.k.shape[3], cache.v.shape[3]) if raw else (cache.D, cache.Dv)
    with _On(dev, stream) as on:
        if out is None:
            out = {"k": torch.empty((T, cache.Hkv, nk), dtype=dtype, device=dev),
                   "v": torch.empty((T, cache.Hkv, nv), dtype=dtype, device=dev)}
        else:
            _expect("out k", out["k"], dtype, (T, cache.Hkv, nk), dev)
            _expect("out v", out["v"], dtype, (T, cache.Hkv, nv), dev)
        _check(nat.fa_cache_read(cache.c, seq.data_ptr(), pos.data_ptr(), T, act, out["k"].data_ptr(),
                                 out["v"].data_ptr(), on.handle))
    return out


def paged_decode(q: torch.Tensor, cache: PagedCache, seq_lens: torch.Tensor, *, scale: float,
                 alibi_slopes: Optional[torch.Tensor] = None, softcap: float = 0.0,
                 sinks: Optional[torch.Tensor] = None, out: Optional[dict] = None,
                 workspace: Optional[Workspace] = None, stream: Optional[torch.cuda.Stream] = None) -> dict:
    """Attention of one new token per sequence: q [B][H][D] (f32, f16 or bf16; may be a view) over the first
    seq_lens [B] (int32) positions of the cache's sequences: {"O": [B][H][Dv] of q's type, "lse": [B][H] f32}.
    ALiBi slopes and sinks (f32 [H]) and the soft cap are those of backward().  A negative length marks a
    padding slot, whose rows are not written."""
    B, H = q.shape[0], q.shape[1]
    dev = cache.device
    act = _act(q.dtype)
    _heads("q", q, cache.B, cache.D, q.dtype, dev)
    _expect("seq_lens", seq_lens, torch.int32, (B,), dev)
    _expect("alibi_slopes", alibi_slopes, torch.float32, (H,), dev)
    _expect("sinks", sinks, torch.float32, (H,), dev)
    with _On(dev, stream) as on:
        ws = (workspace or Workspace(dev)).get(cache.decode_workspace_size(H))
        if out is None:
            out = {"O": torch.empty((B, H, cache.Dv), dtype=q.dtype, device=dev),
                   "lse": torch.empty((B, H), dtype=torch.float32, device=dev)}
        else:
            _expect("out O", out["O"], q.dtype, (B, H, cache.Dv), dev)
            _expect("out lse", out["lse"], torch.float32, (B, H), dev)
        _check(nat.fa_paged_decode(q.data_ptr(), act, q.stride(0), q.stride(1), cache.c, seq_lens.data_ptr(), H, scale,
                                   _ptr(alibi_slopes), softcap, _ptr(sinks), out["O"].data_ptr(), out["lse"].data_ptr(),
                                   ws.data_ptr(), ws.numel(), on.handle))
    return out


def _qk(q, k, N, D, dtype, dev):
    _heads("q", q, N, D, dtype, dev)
    if k is None:
        return 0, nat.fa_qk_views(q.stride(0), q.stride(1), 0, 0)
    _heads("k", k, N, D, dtype, dev)
    return k.shape[1], nat.fa_qk_views(q.stride(0), q.stride(1), k.stride(0), k.stride(1))


def qk_norm_rope(q: torch.Tensor, k: Optional[torch.Tensor], pos: Optional[torch.Tensor], *,
                 wq: Optional[torch.Tensor] = None, wk: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 rope: Optional[torch.Tensor] = None, rope_style: int = nat.FA_ROPE_HALVES, dtype=None,
                 out: Optional[dict] = None, stream: Optional[torch.cuda.Stream] = None) -> dict:
    """RMS norm of every head (weights wq, wk f32 [D]; None: not normalised) and rotation by pos [N]
    (int32) of queries q [N][H][D] and keys k [N][Hkv][D] (f32, f16 or bf16, possibly views of one
    projection; k may be None): {"q", "k"}, contiguous, of dtype (default q's)."""
    N, H, D = q.shape
    dev = q.device
    Hkv, views = _qk(q, k, N, D, q.dtype, dev)
    dtype = q.dtype if dtype is None else dtype
    x_type, y_type = _act(q.dtype), _act(dtype)
    _expect("wq", wq, torch.float32, (D,), dev)
    _expect("wk", wk, torch.float32, (D,), dev)
    r = _rope(rope, rope_style, pos, N, dev)
    with _On(dev, stream) as on:
        if out is None:
            out = {"q": torch.empty((N, H, D), dtype=dtype, device=dev),
                   "k": None if k is None else torch.empty((N, Hkv, D), dtype=dtype, device=dev)}
        else:
            _expect("out q", out["q"], dtype, (N, H, D), dev)
            _expect("out k", out["k"], dtype, (N, Hkv, D), dev)
        _check(nat.fa_qk_norm_rope(q.data_ptr(), _ptr(k), x_type, views, _ptr(wq), _ptr(wk), eps,
                                   None if r is None else pos.data_ptr(), r, N, H, Hkv, D, out["q"].data_ptr(),
                                   _ptr(out["k"]), y_type, on.handle))
    return out


def qk_norm_rope_backward(gq: torch.Tensor, gk: Optional[torch.Tensor], q: torch.Tensor, k: Optional[torch.Tensor],
                          pos: Optional[torch.Tensor], *, wq: Optional[torch.Tensor] = None,
                          wk: Optional[torch.Tensor] = None, eps: float = 1e-6, rope: Optional[torch.Tensor] = None,
                          rope_style: int = nat.FA_ROPE_HALVES, out: Optional[dict] = None,
                          workspace: Optional[Workspace] = None,
                          stream: Optional[torch.cuda.Stream] = None) -> dict:
    """The gradient of qk_norm_rope(): given gq [N][H][D] and gk [N][Hkv][D] (contiguous, e.g. backward()'s dQ
    and dK) and the forward's inputs, {"dq", "dk" of q's type, "dwq", "dwk" f32 [D] (with the weights)}."""
    N, H, D = q.shape
    dev = q.device
    Hkv, views = _qk(q, k, N, D, q.dtype, dev)
    if (gk is None) != (k is None):
        raise FaBackError("gk and k are given together")
    x_type, y_type = _act(q.dtype), _act(gq.dtype)
    _expect("gq", gq, gq.dtype, (N, H, D), dev)
    _expect("gk", gk, gq.dtype, (N, Hkv, D), dev)
    _expect("wq", wq, torch.float32, (D,), dev)
    _expect("wk", wk, torch.float32, (D,), dev)
    r = _rope(rope, rope_style, pos, N, dev)
    with _On(dev, stream) as on:
        if out is None:
            out = {"dq": torch.empty((N, H, D), dtype=q.dtype, device=dev)}
            if k is not None:
                out["dk"] = torch.empty((N, Hkv, D), dtype=q.dtype, device=dev)
            if wq is not None:
                out["dwq"] = torch.empty((D,), dtype=torch.float32, device=dev)
            if wk is not None and k is not None:
                out["dwk"] = torch.empty((D,), dtype=torch.float32, device=dev)
        else:
            _expect("out dq", out["dq"], q.dtype, (N, H, D), dev)
            _expect("out dk", out.get("dk"), q.dtype, (N, Hkv, D), dev)
            _expect("out dwq", out.get("dwq"), torch.float32, (D,), dev)
            _expect("out dwk", out.get("dwk"), torch.float32, (D,), dev)
        ws = (workspace or Workspace(dev)).get(nat.fa_qk_norm_rope_backward_workspace_size(N, H, Hkv, D))
        _check(nat.fa_qk_norm_rope_backward(
            gq.data_ptr(), _ptr(gk), y_type, q.data_ptr(), _ptr(k), x_type, views, _ptr(wq), _ptr(wk), eps,
            None if r is None else pos.data_ptr(), r, N, H, Hkv, D, out["dq"].data_ptr(), _ptr(out.get("dk")),
            _ptr(out.get("dwq")), _ptr(out.get("dwk")), ws.data_ptr(), ws.numel(), on.handle))
    return out
